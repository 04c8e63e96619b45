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
// halves, less 1024 is the code, and one HFMA2 gives lo + s * code, rounded once (2^-11 of
// the value).  K, V and q are scaled by powers of two into fp16's range: the writes keep the
// largest and the smallest size of a unit's groups, and a sequence in which they are 2^24 apart
// is left to wide_rows(), since below that groups would lose bits.  A bf16 q is exact but for
// elements below 2^-26 of the row's largest (off by 2^-35 of that).  P is scaled to at most
// 2^14: its rounding is 2^-11 relative down to 2^-28 of the largest.  The running reference
// (a score of the row) moves only when a score passes it by 6 (in log2), so O is seldom
// rescaled; it, the sum of P, S and O are fp32.
//
// Bound: 4 d flops a pair of row and token.  A tile of 128 tokens and two streams takes 2048
// cycles of products at the tensor cores' rate and as many of exponentials (16 a cycle and
// SM).  Measured (B200): 512 rows at 32768 tokens, 8 KV heads, 32 heads, d = 128: 350 us for
// 273 GFLOP, 780 TFLOP/s, 48% of a library bf16 product; 5400 cycles a tile, tensor pipe
// active 36%.  What bounds it is a stream's own chain: S to P about 2700 cycles (loads from
// TMEM, 128 exponentials a thread, stores), P to the next S 2600 (two groups of eight products
// and three barriers).  Leaving out half of the products (in a copy) saved 6%, and three
// quarters of the softmax and of the conversion 25%.  Tried and slower: a second issuing
// thread (429 us), 16 scores at a time (542), polling instead of suspended waits (684), tiles
// asked into L2 ahead (+10%), registers shared out by role so that 64 scores stay over the
// maximum (408), everything unrolled (instruction cache).
//
// The products' accumulators do not round to nearest: over 7080 products (885 tiles) O shrank by
// 1.0e-4 of itself.  So a stream adds O to fp32 sums in the workspace every 256 tiles, and O starts
// from zero again (a cache of 32768 tokens and less never gets there).
//
// All tiles of all units (sequence, KV head, block of rows) form one list, cut evenly over
// the CTAs.  Tiles behind a block's last position are left out where slots are positions
// (nothing was evicted).  A unit that is cut leaves partial results (O, m, sum of P), which
// kv4_join_kernel adds in the order of the CTAs.
#include <type_traits>

#include "kv4.cuh"

namespace recsa {

namespace {

constexpr int kTok = 128;                 // tokens of a tile
constexpr int kRowsStream = 128;
// Warpgroups 0 and 1: softmax, a stream each; 2 and 3: codes of K and of V to fp16; the last
// warp issues the products.
constexpr int kSoftWarps = 8, kCodeWarp0 = 8, kMmaWarp = 16;
constexpr int kChunkThreads = 17 * 32;
constexpr int kInfo = 4;                  // tiles whose positions are held (see the ring's use)
constexpr uint32_t kNanPar = 0x7fc00000u;   // lo = NaN, s = 0
constexpr float kUp = 8.0f;               // P is scaled by 2^8, and stays below 2^14
constexpr float kMostP = 16384.0f;        // P moves the reference where it passes 2^(kUp + 6)
constexpr float kNoScore = -3e38f;
constexpr int kFlush = 256;               // tiles of a stream whose products O sums up (a power of two)

template <int D>
struct ChunkSmem {
    static constexpr int kSlab = 128 * 128;             // 128 rows of 64 fp16
    static constexpr int kTileBytes = kSlab * (D / 64);
    static constexpr int kQ = 0;                        // [2 streams]
    static constexpr int kK = 2 * kTileBytes;           // [2 stages]
    static constexpr int kV = 4 * kTileBytes;           // [2 stages]
    static constexpr int kRaw = 6 * kTileBytes;         // a tile of the cache as it lies there
    // of the raw tile: codes and parameters of K, V's parameters and positions (for the
    // softmax), codes and parameters of V
    static constexpr int kCodes = kTok * D / 2, kPars = kTok * D / 8;
    static constexpr int kRawKp = kCodes, kRawVp = kCodes + kPars, kRawPos = kCodes + 2 * kPars;
    static constexpr int kRawV = kRawPos + kTok * 4;
    static constexpr int kRawBytes = kRawV + kCodes + kPars;
    static constexpr int kBytes = kRaw + kRawBytes + 1024;
    static_assert(kRawBytes <= kTileBytes, "the second raw tile lies over the second Q");
};

// The list of tiles: sequence b has nrb[b] blocks of RB rows a KV head; block j sees
// tiles_of(b, j) tiles of the cache.  pre: running totals over b.
struct ChunkPlan {
    int64_t pre[RECSA_MAX_BATCH + 1];
    int64_t first[RECSA_MAX_BATCH];       // tokens that the first block's rows see, + 127; -1: all
    int tmax[RECSA_MAX_BATCH];            // tiles of the whole cache
    int nrb[RECSA_MAX_BATCH];
    int wide_rows[RECSA_MAX_BATCH];       // rows of a wide sequence (it has no block here), else 0
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
            const bool wide = c.wide[b] != 0;
            int n_b = (int)kv4_count(qv.counts, b, qv.n, c.status);
            if (n_b > seen) {             // more rows than tokens: none has a position
                set_status(c.status, kStatusBadQuery);
                n_b = 0;
            }
            int rows = n_b - qv.i0;
            rows = rows < 0 ? 0 : rows < qv.w ? rows : qv.w;
            pl.nrb[b] = wide ? 0 : (rows * c.G + RB - 1) / RB;
            pl.wide_rows[b] = wide ? rows * c.G : 0;
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

__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

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
// One thread of a whole warp, the same each time (a commit stands for what its thread issued).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
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
// Waits for the loads before it; names the registers, so that none is used earlier.
__device__ __forceinline__ void ld_done(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                   "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]),
                   "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                   "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                   "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]),
                   "+f"(v[31])
                 :
                 : "memory");
}
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

__device__ __forceinline__ void ld16(uint32_t t, uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
          "=r"(u[14]), "=r"(u[15])
        : "r"(t)
        : "memory");
}

// ---- softmax of 32 scores of a row ----
// Scores of tokens behind position lim become -infinity, in TMEM.  (Not inlined: the few
// tiles that need it must not lengthen the loop.  The roles' loops run side by side, and when
// everything was unrolled the SM's instruction cache missed at 64% of the next level's rate.)
__device__ __noinline__ void hide_scores(uint32_t t, const int32_t* pos, int lim) {
#pragma unroll 1
    for (int k = 0; k < kTok; k += 32) {
        float s[32];
        ld32(t + k, s);
        ld_done(s);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const int4 p = *reinterpret_cast<const int4*>(pos + k + e);
            if (p.x > lim) s[e] = -INFINITY;
            if (p.y > lim) s[e + 1] = -INFINITY;
            if (p.z > lim) s[e + 2] = -INFINITY;
            if (p.w > lim) s[e + 3] = -INFINITY;
        }
        st32(t + k, s);
    }
    st_done();
}
// p = 2^((s - ref) * scale + kUp) as fp16 and its sum in fp32; returns the largest.  The
// difference comes first: at ref it is exactly 0, however large the scores are.
__device__ __forceinline__ float form_p(const float (&s)[32], float scale, float ref, uint32_t (&p)[16],
                                        float2& sum) {
    float most[2] = {0.0f, 0.0f};
    float2 l[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float2 a = add2(make_float2(s[e], s[e + 1]), make_float2(-ref, -ref));
        a = fma2(a, make_float2(scale, scale), make_float2(kUp, kUp));
        a.x = ex2(a.x);
        a.y = ex2(a.y);
        const int h = (e >> 1) & 1;
        l[h] = add2(l[h], a);
        most[h] = fmaxf(most[h], fmaxf(a.x, a.y));
        p[e >> 1] = as_u(__floats2half2_rn(a.x, a.y));
    }
    sum = add2(l[0], l[1]);
    return fmaxf(most[0], most[1]);
}
// Moves the reference of the rows that are `over` to the largest of scores 32 k .. 32 k + 31:
// the sixteens of P that the tile already has, O (where products went into it) and the sum
// are scaled by the factor, and P of these scores is formed and stored.  The products before
// S are done by now: one thread issued both, and S's barrier stands for all it had issued.
struct Moved { float ref, l; };
template <int D>
__device__ __noinline__ Moved move_reference(uint32_t ts, uint32_t to, int k, bool has_o, float rsc,
                                             bool over, float ref, float2 l2) {
    float s[32];
    ld32(ts + k * 32, s);
    ld_done(s);
    float f = 1.0f;
    if (over) {
        float x = s[0];
#pragma unroll
        for (int e = 1; e < 32; ++e) x = fmaxf(x, s[e]);
        f = ex2((ref - x) * rsc);
        ref = x;
    }
    const __half2 h = __float2half2_rn(f);
    __syncwarp();
    st_done();
#pragma unroll 1
    for (int i = 0; i < k; ++i) {
        uint32_t p[16];
        ld16(ts + i * 16, p);
#pragma unroll
        for (int e = 0; e < 16; ++e) p[e] = as_u(__hmul2(as_h2(p[e]), h));
        st16(ts + i * 16, p);
    }
    uint32_t p[16];
    float2 sum;
    form_p(s, rsc, ref, p, sum);
    st16(ts + k * 16, p);
#pragma unroll 1
    for (int i = 0; has_o && i < D; i += 32) {
        ld32(to + i, s);
        ld_done(s);
#pragma unroll
        for (int e = 0; e < 32; ++e) s[e] *= f;
        st32(to + i, s);
    }
    st_done();
    return {ref, fmaf(l2.x + l2.y, f, sum.x + sum.y)};
}
// A row's O of the last kFlush tiles goes to its sums (of the rows of this stream, 128 apart),
// which are `f` times what is there; f = 0: nothing is there.  (O's products are done, as above.)
template <int D>
__device__ __noinline__ void flush_o(uint32_t to, float4* sum, float f) {
#pragma unroll 1
    for (int k = 0; k < D; k += 32) {
        float o[32];
        ld32(to + k, o);
        ld_done(o);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            float4* s = sum + (k + e) / 4 * kRowsStream;
            float4 v = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            if (f != 0.0f) {
                const float4 y = *s;
                v = make_float4(fmaf(f, y.x, v.x), fmaf(f, y.y, v.y), fmaf(f, y.z, v.z), fmaf(f, y.w, v.w));
            }
            *s = v;
        }
    }
}
// Adds f times the sums of dims 32 k .. to the 32 values of O.
__device__ __forceinline__ void add_sums(float (&o)[32], const float4* sum, float f) {
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        const float4 y = sum[e / 4 * kRowsStream];
        o[e] = fmaf(f, y.x, o[e]);
        o[e + 1] = fmaf(f, y.y, o[e + 1]);
        o[e + 2] = fmaf(f, y.z, o[e + 2]);
        o[e + 3] = fmaf(f, y.w, o[e + 3]);
    }
}
// Groups of dims in which a token that the row sees holds NaN.
template <int NG>
__device__ __noinline__ uint32_t nan_groups(const int32_t* pos, const uint32_t* any,
                                            const uint32_t (*bits)[4], int lim) {
    uint32_t out = 0;
    for (int q = 0; q < 4; ++q) {
        if (!any[q]) continue;
        for (int e = 0; e < 32; ++e)
            if (pos[q * 32 + e] <= lim)
                for (int g = 0; g < NG; ++g) out |= ((bits[q][g] >> e) & 1u) << g;
    }
    return out;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, uint32_t* status,
                                       volatile int* failed) {
    if (mbar_wait_bounded(bar, parity, status, *failed ? kWaitPollsAfterFail : kWaitPolls))
        return *failed == 0;
    *failed = 1;
    return false;
}
__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}


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

// A raw tile to fp16 values, by 128 threads: a lane takes a group of 32 dims (16 bytes of
// codes), a warp 32 neighbouring groups, and the upper groups go through their words in
// another order, so that eight lanes' stores lie in eight different bank groups.  Rows at or
// past `rows` become 0, and with `drop` groups of NaN too.
template <int D>
__device__ __forceinline__ void convert(unsigned char* tile, const unsigned char* codes,
                                        const unsigned char* pars, int tid, int rows, float scale,
                                        bool drop) {
    constexpr int NG = D / 32;
#pragma unroll 1
    for (int i = tid; i < kTok * NG; i += 128) {
        const int row = i / NG, g = i % NG;
        const uint4 c = *reinterpret_cast<const uint4*>(codes + i * 16);
        uint32_t par = *reinterpret_cast<const uint32_t*>(pars + i * 4);
        if (row >= rows || (drop && par == kNanPar)) par = 0;
        const __half2 s = __float2half2_rn(kv4_step(par) * scale);
        const __half2 lo = __float2half2_rn(kv4_off(par) * scale);
        const bool swap = (g & 2) != 0;
        const uint32_t w[4] = {swap ? c.z : c.x, swap ? c.w : c.y, swap ? c.x : c.z, swap ? c.y : c.w};
        const int first = g * 4 + (swap ? 2 : 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int ch = (first & ~3) | ((first + k) & 3);
            *reinterpret_cast<uint4*>(tile + chunk_of(row, ch)) = values8(w[k], s, lo);
        }
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


struct ChunkBars {
    uint64_t raw_full[2][2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full;
};

}  // namespace

// What all threads of a CTA know of the unit they work on.
struct ChunkUnit {
    int64_t start;            // the unit's first tile in the list
    int b, h, u;
    int tiles, tile0, T;      // of the unit; the first that this CTA takes, and how many
    int row0, row_end, n_b;   // rows of the sequence (chunk row times G + head of the group)
    int X;                    // products: x = 0, 1, .., of stream x & 1
};

__device__ __forceinline__ void all_threads() {
    __syncwarp();
    asm volatile("bar.sync 0;" ::: "memory");
}

// part: [2 * grid] of: O [D / 4][RB] float4, m [RB], l [RB].
template <int D, bool TWO>
__global__ void __launch_bounds__(kChunkThreads, 1) kv4_chunk_kernel(Kv4View c, Kv4Query qv,
                                                                     Kv4Scratch sc) {
    constexpr int NG = D / 32;
    using Sm = ChunkSmem<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ ChunkPlan pl;
    __shared__ ChunkUnit un;
    __shared__ ChunkBars bars;
    __shared__ __align__(16) int32_t pos_s[kInfo][kTok];
    __shared__ __align__(16) int32_t pos_max[kInfo][4];
    __shared__ uint32_t nan_s[kInfo][4][4];   // [tile][warp's 32 tokens][group of 32 dims]
    __shared__ __align__(16) uint32_t nan_any[kInfo][4];
    __shared__ float join_m[kRowsStream], join_l[kRowsStream];
    __shared__ uint32_t join_nan[kRowsStream];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int failed;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int RB = TWO ? 256 : 128;       // TWO: two blocks of rows; else the streams share them
    constexpr int sh = TWO ? 1 : 0;           // tile of product x: x >> sh

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.raw_full[0][i], 1);
            mbar_init(&bars.raw_full[1][i], 1);
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
    const int64_t at0 = blockIdx.x * quota;
    const int64_t at_end = at0 + quota < total ? at0 + quota : total;

    // All waits are bounded; one that gives up ends the CTA's work.  What is done already
    // costs one instruction.
    auto wait = [&](uint64_t& bar, uint32_t parity) {
        return mbar_test(&bar, parity) || wait_long(&bar, parity, c.status, &failed);
    };
    // The units of this CTA, by every role in its own branch: stage() before the rows of Q are
    // needed, then work().  Uses of the barriers so far give their parities.
    uint32_t n_tiles = 0, n_units = 0;
    auto for_units = [&](auto stage, auto work) {
        int64_t at = at0;
        int b = 0;
        while (at < at_end) {
            if (threadIdx.x == 0) {
                while (pl.pre[b + 1] <= at) ++b;
                int h, rb;
                int64_t start;
                unit_at(pl, b, at - pl.pre[b], h, rb, start);
                un.b = b;
                un.h = h;
                un.u = b * c.Hkv + h;
                un.start = start + pl.pre[b];
                un.tiles = tiles_of(pl, b, rb);
                un.tile0 = (int)(at - un.start);
                const int64_t left = at_end - at;
                un.T = (int)(left < un.tiles - un.tile0 ? left : un.tiles - un.tile0);
                un.n_b = qv.counts ? qv.counts[b] : qv.n;
                const int w_end = qv.i0 + qv.w < un.n_b ? qv.i0 + qv.w : un.n_b;
                un.row0 = qv.i0 * c.G + rb * RB;
                un.row_end = w_end * c.G;
                un.X = un.T << sh;
            }
            all_threads();
            stage();
            all_threads();
            work();
            at += un.T;
            n_tiles += un.T;
            ++n_units;
            tc_before();
            all_threads();
            tc_after();
            if (failed) break;
        }
    };

    if (warp < kSoftWarps) {
        // ---- softmax: a thread a row ----
        const int stream = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + stream * 128, to = tmem + lanes + 256 + stream * 128;
        int lim = -1, row = 0;
        uint32_t s_parity = 0;
        float rsc = 0.0f;
        auto stage = [&] {
            // this thread's row of Q, scaled by a power of two to [2^10, 2^11)
            row = un.row0 + (TWO ? stream * kRowsStream : 0) + r;
            lim = -1;
            unsigned char* qs = smem + Sm::kQ + stream * Sm::kTileBytes;
            const uint4* q = nullptr;    // read twice: the row need not fit the registers
            float mx = 0.0f;
            if (row < un.row_end) {
                const int i = row / c.G, g = row % c.G;
                lim = (int)(c.seen[un.b] - un.n_b + i);
                q = reinterpret_cast<const uint4*>(
                    reinterpret_cast<const __nv_bfloat16*>(qv.q) +
                    (((int64_t)un.b * qv.n + i) * c.Hq + un.h * c.G + g) * D);
#pragma unroll 4
                for (int k = 0; k < D / 8; ++k) {
                    const uint4 v = __ldg(q + k);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[e] << 16)),
                                             fabsf(__uint_as_float(w[e] & 0xffff0000u))));
                }
            }
            const int ek = exponent_of(__uint_as_float(c.kmax[un.u]));
            const int e0 = exponent_of(mx), eq = e0 < -116 ? -116 : e0;
            const float up = pow2i(10 - eq);
            rsc = fmaxf(fminf(c.scale * 1.4426950408889634f * pow2i(eq - 10 + ek - 13), 3e38f), 1e-38f);
#pragma unroll 4
            for (int k = 0; k < D / 8; ++k) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (q != nullptr) v = __ldg(q + k);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
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
                if (TWO || stream == 0) *reinterpret_cast<uint4*>(qs + chunk_of(r, k)) = y;
            }
            fence_async_smem();
        };
        auto work = [&] {
            const int X = un.X, mine = (X - stream + 1) / 2;
            const bool some = __any_sync(kFull, lim >= 0);
            float ref = kNoScore;      // of the exponent, in the products' units
            float sum_ref = kNoScore;  // the same of this row's sums of O
            float4* sum = sc.sum + ((size_t)blockIdx.x * 2 + stream) * (D / 4) * kRowsStream + r;
            float2 l2 = make_float2(0.0f, 0.0f);
            uint32_t nanbits = 0;
            bool ok = true;
            for (int j = 0; j < mine; ++j) {
                const uint32_t slot = (n_tiles + ((2 * j + stream) >> sh)) % kInfo;
                ok = __all_sync(kFull, wait(bars.s_full[stream], s_parity));
                if (!ok) break;
                s_parity ^= 1;
                tc_after();
                if (some && j > 0 && j % kFlush == 0) {
                    if (!in_bounds(c.R / kTok > kFlush, c.status)) break;   // (sums are there)
                    flush_o<D>(to, sum, j > kFlush ? ex2((sum_ref - ref) * rsc) : 0.0f);
                    sum_ref = ref;
                }
                if (some) {
                    const int4 pm = *reinterpret_cast<const int4*>(pos_max[slot]);
                    const uint4 na = *reinterpret_cast<const uint4*>(nan_any[slot]);
                    const int most = max(max(pm.x, pm.y), max(pm.z, pm.w));
                    if (__any_sync(kFull, most > lim && lim >= 0)) hide_scores(ts, pos_s[slot], lim);
                    if (na.x | na.y | na.z | na.w)
                        nanbits |= nan_groups<NG>(pos_s[slot], nan_any[slot], nan_s[slot], lim);
                    // P is formed with the old reference; should one pass kMostP, that moves to
                    // the largest of the 32 (then none can pass it)
#pragma unroll 1
                    for (int k = 0; k < kTok / 32; k += 2) {
                        // 64 scores at a time; after a retry (a call, which does the 32 scores
                        // itself) the others are read again, so that nothing is held over it
                        float a[32], z[32];
                        uint32_t p[16];
                        float2 sum;
                        ld32(ts + k * 32, a);
                        ld32(ts + k * 32 + 32, z);
                        ld_done(a);
                        ld_done(z);
                        bool over = form_p(a, rsc, ref, p, sum) > kMostP;
                        if (__any_sync(kFull, over)) {
                            const Moved to_new = move_reference<D>(ts, to, k, j > 0, rsc, over, ref, l2);
                            ref = to_new.ref;
                            l2 = make_float2(to_new.l, 0.0f);
                            ld32(ts + k * 32 + 32, z);
                            ld_done(z);
                        } else {
                            l2 = add2(l2, sum);
                            st16(ts + k * 16, p);
                        }
                        over = form_p(z, rsc, ref, p, sum) > kMostP;
                        if (__any_sync(kFull, over)) {
                            const Moved to_new = move_reference<D>(ts, to, k + 1, j > 0, rsc, over, ref, l2);
                            ref = to_new.ref;
                            l2 = make_float2(to_new.l, 0.0f);
                        } else {
                            l2 = add2(l2, sum);
                            st16(ts + k * 16 + 16, p);
                        }
                    }
                    st_done();
                }
                tc_before();
                mbar_arrive(&bars.p_full[stream]);
            }
            // ---- results ----
            float l = l2.x + l2.y;
            float m = l == 0.0f ? kKv4MinLog2 : ref * rsc;
            ok = __all_sync(kFull, ok && wait(bars.o_full, n_units & 1));
            tc_after();
            const int64_t cta0 = un.start / quota, cta1 = (un.start + un.tiles - 1) / quota;
            const bool whole = cta0 == cta1;
            const int ev = exponent_of(__uint_as_float(c.vmax[un.u]));
            const bool sums = mine > kFlush;
            const float f_sum = ex2((sum_ref - ref) * rsc);
            float f0 = 1.0f, f1 = 0.0f;
            float4* other = reinterpret_cast<float4*>(smem + Sm::kK);   // [D / 4][128]: K is done
            if (!TWO) {
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
                            ld_done(o);
                            if (sums) add_sums(o, sum + k / 4 * kRowsStream, f_sum);
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
            if ((TWO || stream == 0) && some && ok) {
                const int i = row / c.G, g = row % c.G, rr = row - un.row0;
                const bool live = row < un.row_end && in_bounds(row < qv.n * c.G && rr < RB, c.status);
                const bool any = l > 0.0f || l != l;
                const float inv = any ? pow2i(ev - 13) / l : 0.0f;
                float* part = sc.part + (size_t)(2 * blockIdx.x + (un.tile0 == 0 ? 1 : 0)) * RB * (D + 2);
                __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(qv.out) +
                                     (((int64_t)un.b * qv.n + i) * c.Hq + un.h * c.G + g) * D;
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    ld32(to + k, o);
                    ld_done(o);
                    if (sums) add_sums(o, sum + k / 4 * kRowsStream, f_sum);
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
                if (live && !whole) {
                    part[(size_t)RB * D + rr] = m;
                    part[(size_t)RB * D + RB + rr] = l;
                }
            }
        };
        for_units(stage, work);
    } else if (warp < kMmaWarp) {
        // ---- codes to fp16: one warpgroup K and what the softmax needs, one V ----
        const int tid = threadIdx.x & 127, is_v = (warp - kCodeWarp0) >> 2, wq = warp & 3;
        // raw tiles on their way: the second lies where two blocks have their second Q
        const int deep = TWO ? 1 : 2;
        auto raw_at = [&](uint32_t n) {
            return smem + (deep == 2 && (n & 1) ? Sm::kQ + Sm::kTileBytes : Sm::kRaw);
        };
        auto work = [&] {
            const int u = un.u, T = un.T, tile0 = un.tile0;
            const int64_t L = c.len[un.b];
            const float scale = pow2i(13 - exponent_of(__uint_as_float((is_v ? c.vmax : c.kmax)[u])));
            auto fetch = [&](int t) {
                const uint32_t n = n_tiles + t;
                int64_t row = u * c.R + (int64_t)(tile0 + t) * kTok;
                if (!in_bounds(tile0 + t >= 0 && (int64_t)(tile0 + t + 1) * kTok <= c.R, c.status)) row = 0;
                unsigned char* raw = raw_at(n);
                uint64_t* bar = &bars.raw_full[is_v][n & (deep - 1)];
                if (is_v) {
                    mbar_expect_tx(bar, Sm::kCodes + Sm::kPars);
                    bulk_g2s(raw + Sm::kRawV, c.vc + row * (D / 2), Sm::kCodes, bar);
                    bulk_g2s(raw + Sm::kRawV + Sm::kCodes, c.vp + row * NG, Sm::kPars, bar);
                } else {
                    mbar_expect_tx(bar, Sm::kCodes + 2 * Sm::kPars + kTok * 4);
                    bulk_g2s(raw, c.kc + row * (D / 2), Sm::kCodes, bar);
                    bulk_g2s(raw + Sm::kRawKp, c.kp + row * NG, Sm::kPars, bar);
                    bulk_g2s(raw + Sm::kRawVp, c.vp + row * NG, Sm::kPars, bar);
                    bulk_g2s(raw + Sm::kRawPos, c.pos + row, kTok * 4, bar);
                }
            };
            int asked = 0;
            if (tid == 0)
                for (; asked < deep && asked < T; ++asked) fetch(asked);
            uint64_t *full = is_v ? bars.v_full : bars.k_full, *empty = is_v ? bars.v_empty : bars.k_empty;
            int t = 0;
            for (; t < T; ++t) {
                const uint32_t n = n_tiles + t, st = n & 1;
                const unsigned char* raw = raw_at(n);
                const int64_t left = L - (int64_t)(tile0 + t) * kTok;
                const int rows = left < kTok ? (int)left : kTok;
                const uint32_t used = deep == 2 ? n >> 1 : n;   // of this raw tile's barrier
                if (!wait(bars.raw_full[is_v][n & (deep - 1)], used & 1)) break;
                if (!wait(empty[st], ((n >> 1) & 1) ^ 1)) break;
                if (is_v) {
                    // the rows that see a NaN group learn of it by nan_s; in a product it
                    // would reach all rows
                    convert<D>(smem + Sm::kV + st * Sm::kTileBytes, raw + Sm::kRawV,
                               raw + Sm::kRawV + Sm::kCodes, tid, rows, scale, true);
                } else {
                    const uint32_t slot = n % kInfo;
                    const int32_t p = tid < rows ? reinterpret_cast<const int32_t*>(raw + Sm::kRawPos)[tid]
                                                 : 0x7fffffff;
                    uint32_t bad = 0;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        bad |= (reinterpret_cast<const uint32_t*>(raw + Sm::kRawVp)[tid * NG + g] == kNanPar
                                    ? 1u : 0u) << g;
                    pos_s[slot][tid] = p;
                    const int32_t most = __reduce_max_sync(kFull, p);
                    const bool any = __any_sync(kFull, bad != 0);
                    if (any) {
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const uint32_t mask = __ballot_sync(kFull, (bad >> g) & 1u);
                            if (lane == 0) nan_s[slot][wq][g] = mask;
                        }
                    }
                    if (lane == 0) {
                        pos_max[slot][wq] = most;
                        nan_any[slot][wq] = any;
                    }
                    convert<D>(smem + Sm::kK + st * Sm::kTileBytes, raw, raw + Sm::kRawKp, tid, rows,
                               scale, false);
                }
                fence_async_smem();
                mbar_arrive(&full[st]);
                asm volatile("bar.sync %0, 128;" ::"r"(2 + is_v) : "memory");   // the raw tile is read
                if (tid == 0 && asked < T) fetch(asked++);
            }
            // after a failure: what was asked for lands before the CTA ends
            if (t < T && tid == 0)
                for (; t < asked; ++t)
                    mbar_wait_bounded(&bars.raw_full[is_v][(n_tiles + t) & (deep - 1)],
                                      (deep == 2 ? (n_tiles + t) >> 1 : n_tiles + t) & 1,
                                      c.status, kWaitPollsAfterFail);
        };
        for_units([] {}, work);
    } else {
        // ---- products ----
        const uint64_t q0 = sw128(smem_u32(smem + Sm::kQ), 16), k0 = sw128(smem_u32(smem + Sm::kK), 16),
                       v0 = sw128(smem_u32(smem + Sm::kV), Sm::kSlab);
        constexpr uint32_t kTile16 = Sm::kTileBytes / 16;   // descriptors count 16 bytes
        constexpr uint32_t id_qk = f16_idesc(kTok, false), id_pv = f16_idesc(D, true);
        uint32_t kn = 0, vn = 0, p_parity[2] = {0, 0};      // tiles of K and V used so far
        auto work = [&] {
            // the whole warp goes through the loop, one elected thread issues
            const int X = __shfl_sync(kFull, un.X, 0);
            bool ok = true;
            auto qk = [&](auto stream) {
                constexpr int i = decltype(stream)::value;
                const uint32_t st = kn & 1;
                if (!wait(bars.k_full[st], (kn >> 1) & 1)) return false;
                tc_after();
                if (elect_one()) {
                    const uint64_t qa = q0 + (TWO ? i * kTile16 : 0), ka = k0 + st * kTile16;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int off = (k >> 2) * (Sm::kSlab / 16) + (k & 3) * 2;
                        mma_ss(tmem + i * 128, qa + off, ka + off, id_qk, k > 0);
                    }
                    commit(&bars.s_full[i]);
                    if (!TWO || i) commit(&bars.k_empty[st]);
                }
                __syncwarp();
                if (!TWO || i) ++kn;
                return true;
            };
            auto pv = [&](auto stream, bool first, bool more) {
                constexpr int i = decltype(stream)::value;
                const uint32_t st = vn & 1;
                if (!wait(bars.v_full[st], (vn >> 1) & 1) || !wait(bars.p_full[i], p_parity[i])) return false;
                p_parity[i] ^= 1;
                tc_after();
                if (elect_one()) {
                    const uint64_t va = v0 + st * kTile16;
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k)
                        mma_ts(tmem + 256 + i * 128, tmem + i * 128 + k * 8, va + k * 128, id_pv,
                               k > 0 || !first);
                    if (!TWO || i) commit(&bars.v_empty[st]);
                }
                __syncwarp();
                if (!TWO || i) ++vn;
                return !more || qk(stream);
            };
            const std::integral_constant<int, 0> s0;
            const std::integral_constant<int, 1> s1;
            ok = qk(s0) && (X < 2 || qk(s1));
            for (int x = 0; ok && x < X; x += 2) {
                const bool first = (x / 2) % kFlush == 0;   // O was moved to the sums
                ok = pv(s0, first, x + 2 < X);
                if (ok && x + 1 < X) ok = pv(s1, first, x + 3 < X);
            }
            if (elect_one()) commit(&bars.o_full);
            __syncwarp();
            // after a failure: what was issued is done before TMEM is given back
            if (!ok) mbar_wait_bounded(&bars.o_full, n_units & 1, c.status, kWaitPollsAfterFail);
        };
        for_units([] {}, work);
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// 32 rows of a unit of a wide sequence (kv4_is_wide), in plain fp32: a lane a row.  Tiles of 32
// tokens: a warp forms the scores of four, then every warp the probabilities (the same ones) and
// its eighth of the output's dims; tokens that a row does not see are left out there, as a NaN
// must not reach it.  The next tile's codes are on their way meanwhile.  Such data is not
// expected, so this is short rather than fast, and stands in the join's launch: a launch of the
// other attention kernel cost every call 4 to 6 us.  Measured: 5 rows x 8 sequences at 9001, all
// wide, 1.2 to 3.0 ms (74 us otherwise), 512 rows at 32768 15 ms (0.35).
constexpr int kWideTok = 32, kJoinThreads = 256;
template <int D>
struct WideSmem {
    float4 q[32][D / 4 + 1], x[kWideTok][D / 4];
    float s[kWideTok][32];
    int32_t pos[kWideTok];
};
template <int D>
__device__ __noinline__ void wide_rows(WideSmem<D>& sm, const Kv4View& c, const Kv4Query& qv, int u,
                                       int rel, int rows) {
    constexpr int E = D / 8, NW = kWideTok * (D / 8) / kJoinThreads;   // words of codes a thread
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = u / c.Hkv, h = u % c.Hkv;
    const int n_b = qv.counts ? qv.counts[b] : qv.n;
    const int row = qv.i0 * c.G + rel + lane, row_end = qv.i0 * c.G + rows;
    const int i = row / c.G, g = row % c.G;
    const int64_t L = c.len[b], at = (((int64_t)b * qv.n + i) * c.Hq + h * c.G + g) * D;
    // (rows that are not there see everything, so that whole tiles are seen by all)
    const int lim = row < row_end ? (int)(c.seen[b] - n_b + i) : 0x7ffffffe;
    for (int d = warp * E; d < (warp + 1) * E; ++d)
        reinterpret_cast<float*>(sm.q[lane])[d] =
            row < row_end ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(qv.q)[at + d]) : 0.0f;
    struct Raw { uint32_t code, par; } k[NW], v[NW];
    int32_t pos = 0x7fffffff;
    auto ask = [&](int64_t t0) {
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int y = threadIdx.x + j * kJoinThreads;
            const int64_t slot = u * c.R + t0 + y / (D / 8);     // (R is a multiple of whole tiles)
            const int64_t word = slot * (D / 8) + y % (D / 8), group = slot * (D / 32) + y % (D / 8) / 4;
            k[j] = {reinterpret_cast<const uint32_t*>(c.kc)[word], c.kp[group]};
            v[j] = {reinterpret_cast<const uint32_t*>(c.vc)[word], c.vp[group]};
        }
        if (threadIdx.x < kWideTok)
            pos = t0 + threadIdx.x < L ? c.pos[u * c.R + t0 + threadIdx.x] : 0x7fffffff;
    };
    auto put = [&](const Raw (&raw)[NW]) {
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int y = threadIdx.x + j * kJoinThreads;
            const float s = kv4_step(raw[j].par), lo = kv4_off(raw[j].par);
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = fmaf(s, (float)((raw[j].code >> (4 * e)) & 15u), lo);
            float4* to = &sm.x[y / (D / 8)][y % (D / 8) * 2];
            to[0] = make_float4(z[0], z[1], z[2], z[3]);
            to[1] = make_float4(z[4], z[5], z[6], z[7]);
        }
    };
    const float scale = c.scale * 1.4426950408889634f;
    float o[E], m = kKv4MinLog2, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    ask(0);
#pragma unroll 1
    for (int64_t t0 = 0; t0 < L; t0 += kWideTok) {
        __syncthreads();
        put(k);
        if (threadIdx.x < kWideTok) sm.pos[threadIdx.x] = pos;
        __syncthreads();
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int d = 0; d < D / 4; ++d) {
            const float4 q = sm.q[lane][d];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 x = sm.x[warp * 4 + j][d];
                s[j] = fmaf(q.x, x.x, fmaf(q.y, x.y, fmaf(q.z, x.z, fmaf(q.w, x.w, s[j]))));
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sm.s[warp * 4 + j][lane] = s[j] * scale;
        __syncthreads();
        put(v);
        if (t0 + kWideTok < L) ask(t0 + kWideTok);
        __syncthreads();
        float mn = m;
        bool all = true;
#pragma unroll 8
        for (int j = 0; j < kWideTok; ++j) {
            const bool sees = sm.pos[j] <= lim;
            all &= sees;
            if (sees) mn = fmaxf(mn, sm.s[j][lane]);
        }
        const float f = ex2(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= f;
        auto add = [&](int j) {
            const float p = ex2(sm.s[j][lane] - m);
            l += p;
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const float4 x = sm.x[j][(warp * E + e) / 4];
                o[e] = fmaf(p, x.x, o[e]);
                o[e + 1] = fmaf(p, x.y, o[e + 1]);
                o[e + 2] = fmaf(p, x.z, o[e + 2]);
                o[e + 3] = fmaf(p, x.w, o[e + 3]);
            }
        };
        if (__all_sync(kFull, all)) {
#pragma unroll 8
            for (int j = 0; j < kWideTok; ++j) add(j);
        } else {
#pragma unroll 1
            for (int j = 0; j < kWideTok; ++j)
                if (sm.pos[j] <= lim) add(j);
        }
    }
    if (row >= row_end) return;
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(qv.out) + at + warp * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<__nv_bfloat162*>(out + e) = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
}

// Joins the parts of the units that were cut.  Grid: x = 32 rows, y = unit; a lane a row, a
// warp some of the 8-dim pieces.
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 3) kv4_join_kernel(const __grid_constant__ Kv4View c,
                                                          const __grid_constant__ Kv4Query qv,
                                                          Kv4Scratch sc, int RB, int ctas) {
    __shared__ ChunkPlan pl;
    __shared__ WideSmem<D> wide;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) make_chunk_plan(pl, c, qv, RB, lane);
    __syncthreads();
    const int u = blockIdx.y, b = u / c.Hkv, h = u % c.Hkv;
    const int rel = blockIdx.x * 32, rb = rel / RB, rr = rel % RB + lane;
    if (rel < pl.wide_rows[b]) {
        wide_rows<D>(wide, c, qv, u, rel, pl.wide_rows[b]);
        return;
    }
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
        if (!in_bounds(cta >= 0 && cta < ctas && rr < RB, c.status)) cta = 0;
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
    const size_t smem = ChunkSmem<D>::kBytes;
    cudaError_t e = RB == 256
        ? kv4_launch(kv4_chunk_kernel<D, true>, dim3(kChunkGrid), kChunkThreads, smem, s, c, qv, sc)
        : kv4_launch(kv4_chunk_kernel<D, false>, dim3(kChunkGrid), kChunkThreads, smem, s, c, qv, sc);
    if (e != cudaSuccess) return e;
    return kv4_launch(kv4_join_kernel<D>, dim3((unsigned)((rows + 31) / 32), (unsigned)(c.B * c.Hkv)),
                      kJoinThreads, 0, s, c, qv, sc, RB, kChunkGrid);
}

}  // namespace

size_t kv4_chunk_part_floats(int D, int rows) {
    return (size_t)2 * kChunkGrid * chunk_rows(rows) * (D + 2);
}

size_t kv4_chunk_sum_floats(int D, int64_t R) {
    return R / kTok > kFlush ? (size_t)kChunkGrid * 2 * kRowsStream * D : 0;
}

template <int D>
static cudaError_t prepare_impl() {
    const cudaError_t e = cudaFuncSetAttribute(
        kv4_chunk_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkSmem<D>::kBytes);
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(kv4_chunk_kernel<D, false>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   ChunkSmem<D>::kBytes);
}
cudaError_t kv4_prepare_chunk(int D) { return D == 128 ? prepare_impl<128>() : prepare_impl<64>(); }

cudaError_t kv4_launch_chunk(const Kv4View& c, const Kv4Query& qv, const Kv4Scratch& sc, cudaStream_t s) {
    NvtxRange nv("recsa kv4 chunk");
    return c.D == 128 ? chunk_impl<128>(c, qv, sc, s) : chunk_impl<64>(c, qv, sc, s);
}

}  // namespace recsa
