// Attention over the 4-bit KV cache, for single tokens and for chunks:
//
//   o_r = sum_t p_rt V_t,   p_rt = exp(scale q_r . K_t) / sum_t' exp(scale q_r . K_t')
//
// with K_t, V_t = lo + s * code in groups of 32 dims (kv4.cuh), over the tokens that row
// r may see.  Decode reads 160 bytes a token and KV head (d = 128) and computes 4 d G
// flops on them, so it is bound by the cache read; dequantising every code to a float
// would cost more issue slots than the bytes take to arrive, so no code is dequantised:
//
//   * Codes are the operands of mma.sync.m16n8k16 (fp16 in, fp32 accumulators).  A nibble in
//     place in a 16-bit half is a subnormal fp16 number, code * 2^-24 (or code * 2^-20 for the
//     nibble above it), exact: `word & 0x000f000f` is two operand elements.  The products
//     of subnormal operands are aligned by their unnormalised exponent, which leaves about
//     18 bits of a sum: enough beside bf16 (2^-9), used there for K.  Elsewhere the nibble
//     is joined to an exponent (1024 + code) and 1032 subtracted: code - 8, a normal number.
//   * Scores: S[16 tokens x 8 columns] per group of 32 dims from two MMAs with the codes
//     as A (ldmatrix of the packed rows) and q as B, then s and lo enter in fp32:
//     S += s_tg * (code . q)_tg + lo_tg * (sum of q over g).
//   * Output: O^T[32 dims x 8 columns] += codes^T P' with P' = p_rt * s_tg as B.
//     ldmatrix.trans on 16-bit units (four codes) puts tokens 2t, 2t + 1 of four dims into
//     one register, so the same masks give the A operands; p's accumulator layout becomes
//     B's by one movmatrix.  Codes enter as code - 8: codes are never negative, so without
//     that O would be a small difference of two large sums.  sum p (lo + 8 s) is kept in
//     fp32 beside it.
//
// Precision.  q enters as fp16 scaled by a power of two to [2^10, 2^11): a bf16 q is exact
// there but for elements below 2^-23 of the row's largest (off by 2^-31 of that).  P' enters as
// fp16, off by at most 2^-11 relative, less than bf16's own 2^-8 of the output.  fp32 tensors
// use two fp16 columns a row for q and for P' (high and low part, 22 bits; the low part of P'
// is scaled by 2^11, so that it keeps its bits where P' itself is below fp16's normal range).
// The softmax maximum, its sum and all accumulators are fp32.  The products' own accumulators do
// not round to nearest: summed up in them, the codes' share drifts, and what is left beside the
// offsets' share may be a thousandth of it (16 sequences of 524288 x 16 KV heads in bf16: 3.1e-3
// of the output instead of 1.67e-3; fp32, 700000 tokens: 2e-4 instead of 2e-6).  So each
// product's result is added to O, which costs 4 x 524288 12 us of 711.
//
// Each row and group of dims has its own scale of P' (`up`): p s may span any range, and what
// falls below fp16 is less than 2^-30 of the row's and group's largest p s so far.  So a huge
// value hurts no row that gives it no weight, and a heavy token of tiny value no background
// behind it.  A P' that passes 2^14 lowers its scale and O with it; where the running maximum
// moves, O as a sum falls, which raises the scale instead.  (One scale a unit, from the largest
// value ever written, took 667 us instead of 689 at 4 x 524288 and 10.0 instead of 10.9 at 37
// tokens, but lost every value below 2^-24 of that one.)
//
// Work.  A unit is (sequence, KV head, block of 8 rows; fp32: 4, 8 or 16); its cache is cut into tiles
// of 32 tokens.  All tiles of all units form one list, cut evenly over a persistent grid
// (so ragged batches balance); a CTA's warps take its tiles in turn, each with its own ring
// of TMA stages, running maximum and accumulators, and meet only at the end of a unit.  A
// unit cut over several CTAs is joined by the last of each 16 and then by the last of those
// (one CTA joining all 74 of a unit took longer than the unit).
//
// Measured (B200): decode of 4 x 524288 tokens, 8 KV heads, 32 heads, d = 128: 711 us for
// 2684 MB, 3.8 TB/s, 58% of a plain copy's rate (699 to 723 from box to box).  540 instructions a
// warp for 16 tokens of K and V would take 1.2 times the copy's time if one were issued in every
// cycle; 62% of the cycles issue one and the busiest pipe (masks and conversions) is half used,
// so what bounds it is the latency of a warp's one chain at four warps a scheduler.  131072
// tokens of one sequence: 64 us, of which the start, the plan and the joins are about 20.
#include <type_traits>

#include "kv4.cuh"

namespace recsa {

namespace {

constexpr int kTile = 32;            // tokens of a warp's stage
constexpr int kAttendWarps = 4;
constexpr int kAttendThreads = kAttendWarps * 32;
constexpr int kStagesKv4 = 2;
constexpr int kGridMax = 148 * 4;
constexpr int kJoin = 16;            // partial results that one CTA joins
constexpr float kSlack = 6.0f;       // p may reach 2^6 before the running maximum moves
constexpr int kMostUpLog2 = 120;     // largest scale of P' (a power of two), and the first
constexpr int kMostLog2 = 14;        // P' moves its scale where it passes 2^14 ..
constexpr float kSetUp = 0x1p-8f;    // .. which is set so that the largest P' is 2^5 to 2^6
constexpr float kLowUp = 2048.0f;    // fp32 tensors: scale of the low part of P' (its own column)

template <int D>
struct Stage {
    static constexpr int kCodes = kTile * D / 2;
    static constexpr int kPars = kTile * D / 8;
    static constexpr int kK = 0, kV = kCodes, kKp = 2 * kCodes, kVp = 2 * kCodes + kPars;
    static constexpr int kPos = 2 * kCodes + 2 * kPars, kW = kPos + kTile * 4;
    // a multiple of the swizzle pattern (512 bytes for 64-byte rows, 256 for 32-byte)
    static constexpr int kBytes = ((kW + kTile * 4) + 511) / 512 * 512;
};

// Byte offset of 16-byte chunk `ch` (one group) of row r in a swizzled tile.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int ch) {
    if constexpr (D == 128) return (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
    return (uint32_t)(r * 32 + ((ch ^ ((r >> 2) & 1)) << 4));
}

__device__ __forceinline__ void tma_rows(void* dst, const CUtensorMap* m, int row, int unit,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(m), "r"(0), "r"(row), "r"(unit), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero accumulators (which then need no registers).
__device__ __forceinline__ void mma16816_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1) {
    const float z = 0.0f;
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z));
}
__device__ __forceinline__ void mma16816_bf16_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                uint32_t a3, uint32_t b0, uint32_t b1) {
    const float z = 0.0f;
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z));
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}
// code - 8 of a nibble of both halves as normal fp16 numbers: the low nibble joined to 1024,
// less 1032; the nibble above it joined to 64, less 72.  The exponents come from registers
// (an instruction takes one immediate, the mask).
struct Centre {
    uint32_t lo, hi;
    __device__ __forceinline__ Centre() {
        asm volatile("mov.b32 %0, 0x64006400;" : "=r"(lo));
        asm volatile("mov.b32 %0, 0x54005400;" : "=r"(hi));
    }
    __device__ __forceinline__ uint32_t low(uint32_t x) const {
        uint32_t y;
        asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;\n\tadd.rn.f16x2 %0, %0, %3;"
            : "=r"(y) : "r"(x), "r"(lo), "r"(0xe408e408u));
        return y;
    }
    __device__ __forceinline__ uint32_t high(uint32_t x) const {
        uint32_t y;
        asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;\n\tadd.rn.f16x2 %0, %0, %3;"
            : "=r"(y) : "r"(x), "r"(hi), "r"(0xd480d480u));
        return y;
    }
};

// The largest P' of a lane: fp16 pairs as integers (no P' is negative), fp32 tensors' high parts.
template <int T>
struct Largest {
    uint32_t x = 0;
    float y = 0.0f;
    __device__ __forceinline__ void add(uint32_t a, uint32_t b) { x = __vimax3_u16x2(x, a, b); }
    __device__ __forceinline__ void add(float a, float b) { y = fmaxf(y, fmaxf(a, b)); }
    __device__ __forceinline__ bool over() const {
        if (T == 2) return y > (float)(1 << kMostLog2);
        constexpr uint32_t most = (uint32_t)(kMostLog2 + 15) << 10;   // as fp16
        return x >= (most + 1u) << 16 || (x & 0xffffu) > most;
    }
};

// Scales row e of a lane in the accumulators of one group's output.
template <int T>
__device__ __forceinline__ void scale_row(float (&o)[2][4], int e, float f) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int z = 0; z < 4; ++z)
            if (T == 2 || (z & 1) == e) o[k][z] *= f;
}

// Rows of a column set (8 MMA columns): one column a row, or a high and a low column.
template <int T> constexpr int rows_of_set() { return 8 / T; }
// Rows whose columns a lane holds in an accumulator.
template <int T> constexpr int rows_of_lane() { return 2 / T; }

// The block of rows a unit's MMA columns hold, staged once per unit in shared memory.
template <int D, int T, int NCS>
struct Rows {
    static constexpr int NG = D / kKv4Group;
    static constexpr int RB = NCS * 8 / T;
    uint4 frag[NCS][NG][32];         // B operands of the two MMAs of a group, by lane
    float sum[RB][NG];               // fp32 tensors: sums of q over a group
    uint2 off[32];                   // bf16: the same sums as the offsets' B operand, by lane
    float scale[RB];                 // accumulator -> score in log2 units
    int lim[RB];                     // last position the row sees, -1: no row
};

// Stages rows row0 .. row0 + blocks * RB - 1 of (b, h) (row = chunk row * G + head of the group)
// into as many blocks.  A warp takes a row in turn, four loaded before the first is used (one
// at a time, staging 128 rows took longer than the weights' products over them); `n_b` rows
// of the sequence are in use, positions end at `seen`.
template <int D, int T, int NCS>
__device__ void stage_rows(Rows<D, T, NCS>* blocks_of, int blocks, const Kv4View& c, const Kv4Query& qv,
                           int b, int h, int row0, int row_end, int n_b, int64_t seen, int warp,
                           int nwarps, int lane) {
    constexpr int RB = NCS * 8 / T, E = D / 32, NG = D / kKv4Group;
    using TI = typename std::conditional<T == 1, __nv_bfloat16, float>::type;
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int r0 = warp; r0 < blocks * RB; r0 += kBatch * nwarps) {
    float q[kBatch][E];              // dims lane * E ..: a group is 32 / E lanes
    int at[kBatch];                  // last position the row sees, -1: no row
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int row = row0 + r0 + k * nwarps, i = row / c.G, g = row % c.G;
        const bool live = r0 + k * nwarps < blocks * RB && row < row_end && i < n_b;
        at[k] = live ? (int)(seen - n_b + i) : -1;
#pragma unroll
        for (int e = 0; e < E; ++e) q[k][e] = 0.0f;
        if (live) {
            const TI* p = reinterpret_cast<const TI*>(qv.q) +
                          (((int64_t)b * qv.n + i) * c.Hq + h * c.G + g) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) q[k][e] = (float)p[e];
        }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        if (r0 + k * nwarps >= blocks * RB) break;
        Rows<D, T, NCS>& rs = blocks_of[(r0 + k * nwarps) / RB];
        const int r = (r0 + k * nwarps) % RB;
        float(&x)[E] = q[k];
        float mx = 0.0f, sum = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        const int e0 = exponent_of(mx), ex = e0 < -116 ? -116 : e0;
        const float up = pow2i(10 - ex);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] *= up;
            sum += x[e];
        }
        // the sum over the group's 32 / E lanes
#pragma unroll
        for (int o = 1; o < 32 / E; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (lane % (32 / E) == 0) {
            const int j = lane / (32 / E);
            if constexpr (T == 1) {
                // three bf16 parts (24 bits) meet one bf16 offset
                const float x0 = sum * 0x1p-24f;
                const __nv_bfloat16 h = __float2bfloat16_rn(x0);
                const float x1 = x0 - __bfloat162float(h);
                const __nv_bfloat16 m = __float2bfloat16_rn(x1);
                const __nv_bfloat162 a = __halves2bfloat162(h, m);
                const __nv_bfloat162 z = __floats2bfloat162_rn(x1 - __bfloat162float(m), 0.0f);
                rs.off[r * 4 + j] = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                               *reinterpret_cast<const uint32_t*>(&z));
            } else {
                rs.sum[r][j] = sum;
            }
        }
        if (T == 1 && NG == 2 && lane >= 2 && lane < 4) rs.off[r * 4 + lane] = make_uint2(0, 0);
        if (lane == 0) {
            rs.scale[r] = fminf(c.scale * 1.4426950408889634f * pow2i(ex - 10) * (T == 1 ? 0x1p24f : 1.0f), 3e38f);
            rs.lim[r] = at[k];
        }
        // dim 8t + k of a group (k < 8) sits in 16-bit unit (k >> 1 with the pairs
        // (0,4), (1,5), (2,6), (3,7)) of lane (column, t); odd pairs meet codes * 16
        __half* f = reinterpret_cast<__half*>(&rs.frag[r / (8 / T)][0][0]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int dim = lane * E + e, grp = dim / 32, t = (dim / 8) & 3, d8 = dim & 7;
            const float y = T == 1 && (d8 & 1) ? x[e] * 0.0625f : x[e];
            const int reg = d8 & 3, half = d8 >> 2;
            if constexpr (T == 1) {
                const int l = (r & 7) * 4 + t;
                f[((grp * 32 + l) * 4 + reg) * 2 + half] = __float2half_rn(y);
            } else {
                const int l = (r & 3) * 2 * 4 + t;
                const __half hi = __float2half_rn(y);
                f[((grp * 32 + l) * 4 + reg) * 2 + half] = hi;
                f[((grp * 32 + l + 4) * 4 + reg) * 2 + half] = __float2half_rn(y - __half2float(hi));
            }
        }
    }
    }
}

template <int NG>
__device__ __forceinline__ void load_pars(uint32_t (&p)[NG], const unsigned char* base, int row) {
    if constexpr (NG == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(base + row * 16);
        p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(base + row * 8);
        p[0] = v.x; p[1] = v.y;
    }
}

// Scores of 16 tokens (rows r0 .. r0 + 15 of a tile at `st`) against every column set, in
// the rows' scale: sc[c][2 * e + k] for the lane's row e and token g (k = 0) or g + 8.
// bf16 (one column set): lo . sum(q) is a product of its own, the K dimension the groups, four
// places each: the offset stands in all four (bf16, exact), the sum's parts in three.
template <int D, int T, int NCS>
__device__ __forceinline__ void scores16(float (&sc)[NCS][2 * (2 / T)], const unsigned char* st,
                                         const Rows<D, T, NCS>& rs,
                                         const uint4 (&qreg)[NCS == 1 ? D / 32 : 1],
                                         const float (&qsum)[NCS == 1 ? 2 / T : 1][D / 32],
                                         uint2 qoff, const Centre& ctr, int r0, int lane) {
    constexpr int NG = D / kKv4Group, RL = 2 / T;
    static_assert(T == 2 || NCS == 1, "bf16 rows past one column set go to the chunk kernel");
    const int t = lane & 3, g = lane >> 2;
    const uint32_t kc = smem_u32(st + Stage<D>::kK);
    uint32_t p0[NG], p1[NG];
    load_pars<NG>(p0, st + Stage<D>::kKp, r0 + g);
    load_pars<NG>(p1, st + Stage<D>::kKp, r0 + g + 8);
    if constexpr (T == 1) {
        const uint32_t* par = reinterpret_cast<const uint32_t*>(st + Stage<D>::kKp) + t % NG;
        const uint32_t x0 = __byte_perm(par[(r0 + g) * NG], 0, 0x3232);
        const uint32_t x1 = __byte_perm(par[(r0 + g + 8) * NG], 0, 0x3232);
        float acc[4];
        mma16816_bf16_0(acc, x0, x1, x0, x1, qoff.x, qoff.y);
        sc[0][0] = acc[0];
        sc[0][2] = acc[1];
        sc[0][1] = acc[2];
        sc[0][3] = acc[3];
    } else {
#pragma unroll
        for (int c = 0; c < NCS; ++c)
#pragma unroll
            for (int e = 0; e < 2 * RL; ++e) sc[c][e] = 0.0f;
    }
#pragma unroll
    for (int j2 = 0; j2 < NG; j2 += 2) {
        uint32_t w[4];   // tokens 0-7 and 8-15 of group j2, then of j2 + 1
        ldsm4(w, kc + chunk_at<D>(r0 + (lane & 15), j2 + (lane >> 4)));
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            const int j = j2 + jj;
            const uint32_t wa = w[2 * jj], wb = w[2 * jj + 1], va = wa >> 8, vb = wb >> 8;
            const float s0 = kv4_step(p0[j]), s1 = kv4_step(p1[j]);
            if constexpr (T == 1) {
                float acc[4];
                mma16816_0(acc, wa & 0x000f000fu, wb & 0x000f000fu, wa & 0x00f000f0u, wb & 0x00f000f0u,
                           qreg[j].x, qreg[j].y);
                mma16816(acc, va & 0x000f000fu, vb & 0x000f000fu, va & 0x00f000f0u, vb & 0x00f000f0u,
                         qreg[j].z, qreg[j].w);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sc[0][2 * e] = fmaf(s0, acc[e], sc[0][2 * e]);
                    sc[0][2 * e + 1] = fmaf(s1, acc[2 + e], sc[0][2 * e + 1]);
                }
            } else {
                // fp32: centred codes, so that the two terms of a score stay small
                const uint32_t a[8] = {ctr.low(wa), ctr.low(wb), ctr.high(wa), ctr.high(wb),
                                       ctr.low(va), ctr.low(vb), ctr.high(va), ctr.high(vb)};
                const float o0 = fmaf(8.0f, s0, kv4_off(p0[j])), o1 = fmaf(8.0f, s1, kv4_off(p1[j]));
#pragma unroll
                for (int c = 0; c < NCS; ++c) {
                    uint4 q;
                    if constexpr (NCS == 1) q = qreg[j]; else q = rs.frag[c][j][lane];
                    float acc[4];
                    mma16816_0(acc, a[0], a[1], a[2], a[3], q.x, q.y);
                    mma16816(acc, a[4], a[5], a[6], a[7], q.z, q.w);
                    const float qs = NCS == 1 ? qsum[0][j] : rs.sum[c * 4 + t][j];
                    sc[c][0] = fmaf(s0, acc[0] + acc[1], fmaf(o0, qs, sc[c][0]));
                    sc[c][1] = fmaf(s1, acc[2] + acc[3], fmaf(o1, qs, sc[c][1]));
                }
            }
        }
    }
}

// The warps' stages; at the end of a unit their partial outputs lie over them.
template <int D, int RB>
__host__ __device__ constexpr size_t ring_bytes() {
    const size_t stages = (size_t)kAttendWarps * kStagesKv4 * Stage<D>::kBytes;
    const size_t partials = (size_t)kAttendWarps * RB * D * sizeof(float);
    return stages > partials ? stages : partials;
}
// CTAs an SM holds: 128 registers a thread carry one column set, 255 four.
template <int NCS> constexpr int ctas_per_sm() { return NCS == 1 ? 4 : NCS == 2 ? 3 : 2; }

// The tiles of a launch: sequence b has nrb[b] blocks of rows a KV head, each over
// tiles[b] tiles of its cache; `pre` are their running totals over b.
struct Plan {
    int64_t pre[RECSA_MAX_BATCH + 1];
    int tiles[RECSA_MAX_BATCH];
    int nrb[RECSA_MAX_BATCH];
};

__device__ __forceinline__ void make_plan(Plan& pl, const Kv4View& c, const Kv4Query& qv, int RB,
                                          bool one_block, bool chunk, int lane) {
    // warp 0: two sequences a lane
    int64_t v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int b = 2 * lane + k;
        v[k] = 0;
        if (b < c.B) {
            const int64_t L = c.len[b];
            int n_b = (int)kv4_count(qv.counts, b, qv.n, c.status);
            if (chunk && n_b > c.seen[b]) {   // more rows than tokens: none has a position
                set_status(c.status, kStatusBadQuery);
                n_b = 0;
            }
            int rows = n_b - qv.i0;
            rows = rows < 0 ? 0 : rows < qv.w ? rows : qv.w;
            const int nrb = one_block ? (rows > 0 ? 1 : 0) : (rows * c.G + RB - 1) / RB;
            // a block whose sequence is empty still has its zero rows to write
            const int tiles = (int)((L + kTile - 1) / kTile) + (L == 0 ? 1 : 0);
            pl.tiles[b] = tiles;
            pl.nrb[b] = nrb;
            v[k] = (int64_t)c.Hkv * nrb * tiles;
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

}  // namespace

template <int D, int T, int NCS, bool CHUNK>
__global__ void __launch_bounds__(kAttendThreads, ctas_per_sm<NCS>()) kv4_attend_kernel(
    Kv4View c, Kv4Query qv, Kv4Scratch sc_, const __grid_constant__ Kv4Maps maps) {
    constexpr int NG = D / kKv4Group, RB = NCS * 8 / T, RL = 2 / T, RS = 8 / T;
    using St = Stage<D>;
    using RowsT = Rows<D, T, NCS>;
    using TI = typename std::conditional<T == 1, __nv_bfloat16, float>::type;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* ring = smem;
    RowsT& rs = *reinterpret_cast<RowsT*>(smem + ring_bytes<D, RB>());
    __shared__ Plan pl;
    __shared__ uint64_t bars[kAttendWarps][kStagesKv4];
    __shared__ float red_m[kAttendWarps][RB], red_l[kAttendWarps][RB];
    __shared__ int last_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    if (threadIdx.x == 0) {
        for (int w = 0; w < kAttendWarps; ++w)
            for (int s = 0; s < kStagesKv4; ++s) mbar_init(&bars[w][s], 1);
        mbar_fence_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) make_plan(pl, c, qv, RB, false, CHUNK, lane);
    __syncthreads();
    const int64_t total = pl.pre[c.B];
    int64_t quota = (total + gridDim.x - 1) / gridDim.x;
    if (quota < kAttendWarps) quota = kAttendWarps;   // one tile a warp at least
    int64_t at = blockIdx.x * quota;
    int64_t at_end = at + quota < total ? at + quota : total;
    uint32_t phase = 0;                                // bit s: parity of stage s
    bool alive = true;                                 // no wait of this warp gave up
    unsigned char* my_ring = ring + warp * kStagesKv4 * St::kBytes;
    const Centre ctr;

    int b = 0;
    while (at < at_end) {
        while (pl.pre[b + 1] <= at) ++b;
        const int tiles = pl.tiles[b], nrb = pl.nrb[b];
        const int64_t in_b = at - pl.pre[b];
        const int64_t uu = in_b / tiles;               // (h, block) of sequence b
        const int tile0 = (int)(in_b - uu * tiles);
        const int tile1 = (int)(at_end - at < tiles - tile0 ? at_end - at + tile0 : tiles);
        const int h = (int)(uu / nrb), rb = (int)(uu % nrb);
        const int u = b * c.Hkv + h;
        const int64_t L = c.len[b];
        const int n_b = qv.counts ? qv.counts[b] : qv.n;
        const int row0 = qv.i0 * c.G + rb * RB;
        const int w_end = qv.i0 + qv.w < n_b ? qv.i0 + qv.w : n_b;
        const int row_end = w_end * c.G;

        auto fetch = [&](int tile, int s) {
            unsigned char* st = my_ring + s * St::kBytes;
            uint64_t* bar = &bars[warp][s];
            int64_t r = (int64_t)tile * kTile;
            if (!in_bounds(r >= 0 && r + kTile <= c.R, c.status)) r = 0;
            mbar_expect_tx(bar, 2 * St::kCodes + 2 * St::kPars + (CHUNK ? kTile * 4 : 0));
            tma_rows(st + St::kK, &maps.k, (int)r, u, bar);
            tma_rows(st + St::kV, &maps.v, (int)r, u, bar);
            bulk_g2s(st + St::kKp, c.kp + (u * c.R + r) * NG, St::kPars, bar);
            bulk_g2s(st + St::kVp, c.vp + (u * c.R + r) * NG, St::kPars, bar);
            if (CHUNK) bulk_g2s(st + St::kPos, c.pos + u * c.R + r, kTile * 4, bar);
        };
        const int mine = L > 0 ? (tile1 - tile0 - warp + kAttendWarps - 1) / kAttendWarps : 0;
        if (lane == 0 && alive)
            for (int s = 0; s < kStagesKv4 && s < mine; ++s) fetch(tile0 + warp + s * kAttendWarps, s);
        stage_rows<D, T, NCS>(&rs, 1, c, qv, b, h, row0, row_end, n_b, c.seen[b], warp, kAttendWarps, lane);
        __syncthreads();

        float O[NCS][NG][2][4], bias[NCS][RL][NG], m[NCS][RL], l[NCS][RL], rsc[NCS][RL];
        float up[NCS][RL][NG];                         // O is `up` (2^e) times the sum of p s code
        int lim[NCS][RL];
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
#pragma unroll
            for (int j = 0; j < NG; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[cs][j][k][e] = 0.0f;
#pragma unroll
            for (int e = 0; e < RL; ++e) {
                m[cs][e] = kKv4MinLog2;
                l[cs][e] = 0.0f;
                rsc[cs][e] = rs.scale[cs * RS + t * RL + e];
                lim[cs][e] = rs.lim[cs * RS + t * RL + e];
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    bias[cs][e][j] = 0.0f;
                    up[cs][e][j] = pow2i(kMostUpLog2);
                }
            }
        }
        uint4 qreg[NCS == 1 ? NG : 1];
        float qsum[NCS == 1 ? RL : 1][NG];
        if constexpr (NCS == 1) {
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                qreg[j] = rs.frag[0][j][lane];
#pragma unroll
                for (int e = 0; e < RL; ++e) qsum[e][j] = T == 2 ? rs.sum[t * RL + e][j] : 0.0f;
            }
        }
        const uint2 qoff = rs.off[lane];

        for (int it = 0; it < mine; ++it) {
            const int s = it % kStagesKv4;
            const int tile = tile0 + warp + it * kAttendWarps;
            if (!alive) break;
            if (!__all_sync(kFull, mbar_wait_bounded(&bars[warp][s], (phase >> s) & 1u, c.status))) {
                alive = false;
                break;
            }
            phase ^= 1u << s;
            const unsigned char* st = my_ring + s * St::kBytes;
            const uint32_t sa = smem_u32(st);
            const bool tail = (int64_t)(tile + 1) * kTile > L;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int r0 = half * 16;
                const int64_t tok = (int64_t)tile * kTile + r0 + g;
                if (tail && tok - g >= L) break;       // nothing in this half (uniform)
                uint32_t p0[NG], p1[NG];
                float sc[NCS][2 * RL];
                scores16<D, T, NCS>(sc, st, rs, qreg, qsum, qoff, ctr, r0, lane);
                load_pars<NG>(p0, st + St::kVp, r0 + g);
                load_pars<NG>(p1, st + St::kVp, r0 + g + 8);
                int pos0 = -1, pos1 = -1;
                if (CHUNK) {
                    pos0 = *reinterpret_cast<const int*>(st + St::kPos + (r0 + g) * 4);
                    pos1 = *reinterpret_cast<const int*>(st + St::kPos + (r0 + g + 8) * 4);
                }
                if (tail) {
                    // rows past the length: whatever they hold must not enter a product
                    if (tok >= L) {
                        pos0 = 0x7fffffff;
#pragma unroll
                        for (int j = 0; j < NG; ++j) p0[j] = 0;
                    }
                    if (tok + 8 >= L) {
                        pos1 = 0x7fffffff;
#pragma unroll
                        for (int j = 0; j < NG; ++j) p1[j] = 0;
                    }
                }
                bool grow = false;
#pragma unroll
                for (int cs = 0; cs < NCS; ++cs)
#pragma unroll
                    for (int e = 0; e < RL; ++e) {
                        // (rounded on its own: the weights' kernel forms the same bits)
                        sc[cs][2 * e] = __fmul_rn(sc[cs][2 * e], rsc[cs][e]);
                        sc[cs][2 * e + 1] = __fmul_rn(sc[cs][2 * e + 1], rsc[cs][e]);
                        if (CHUNK || tail) {
                            const int lm = CHUNK ? lim[cs][e] : 0x7ffffffe;
                            if (pos0 > lm) sc[cs][2 * e] = -INFINITY;
                            if (pos1 > lm) sc[cs][2 * e + 1] = -INFINITY;
                        }
                        grow |= fmaxf(sc[cs][2 * e], sc[cs][2 * e + 1]) > m[cs][e] + kSlack;
                    }
                if (__any_sync(kFull, grow)) {
                    const bool empty = it == 0 && half == 0;   // no sums yet
#pragma unroll
                    for (int cs = 0; cs < NCS; ++cs)
#pragma unroll
                        for (int e = 0; e < RL; ++e) {
                            float x = fmaxf(sc[cs][2 * e], sc[cs][2 * e + 1]);
                            x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
                            // by a whole number, so that every scaling below is exact
                            const float mn = fmaxf(m[cs][e], ceilf(x));
                            const int k = (int)fminf(mn - m[cs][e], 1000.0f);
                            const float f = pow2z(-k);
                            m[cs][e] = mn;
                            if (empty) continue;
                            l[cs][e] *= f;
#pragma unroll
                            for (int j = 0; j < NG; ++j) {
                                bias[cs][e][j] *= f;
                                // O falls by f as a sum: its scale rises, O stays, up to a limit
                                const int y = exponent_of(up[cs][e][j]) + k;
                                if (y > kMostUpLog2) scale_row<T>(O[cs][j], e, pow2z(kMostUpLog2 - y));
                                up[cs][e][j] = pow2i(y < kMostUpLog2 ? y : kMostUpLog2);
                            }
                        }
                }
#pragma unroll
                for (int cs = 0; cs < NCS; ++cs)
#pragma unroll
                    for (int e = 0; e < RL; ++e) {
                        sc[cs][2 * e] = ex2(sc[cs][2 * e] - m[cs][e]);
                        sc[cs][2 * e + 1] = ex2(sc[cs][2 * e + 1] - m[cs][e]);
                        l[cs][e] += sc[cs][2 * e] + sc[cs][2 * e + 1];
                    }
                // P' and the offsets' share.  (Scale times p first: a step alone may pass fp32,
                // and p = 0 must stay 0.)
                uint32_t b0[NCS][NG], b1[NCS][NG], nan0 = 0, nan1 = 0;
                auto form = [&] {
                    Largest<T> most;
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        const float s0 = kv4_step(p0[j]), s1 = kv4_step(p1[j]);
#pragma unroll
                        for (int cs = 0; cs < NCS; ++cs) {
                            const float u0 = up[cs][0][j], x0 = sc[cs][0] * u0 * s0, x1 = sc[cs][1] * u0 * s1;
                            if constexpr (T == 1) {
                                const float u1 = up[cs][1][j];
                                b0[cs][j] = pack_h2(x0, sc[cs][2] * u1 * s0);
                                b1[cs][j] = pack_h2(x1, sc[cs][3] * u1 * s1);
                                most.add(b0[cs][j], b1[cs][j]);
                            } else {
                                const float h0 = __half2float(__float2half_rn(x0));
                                const float h1 = __half2float(__float2half_rn(x1));
                                b0[cs][j] = pack_h2(h0, (x0 - h0) * kLowUp);
                                b1[cs][j] = pack_h2(h1, (x1 - h1) * kLowUp);
                                most.add(h0, h1);
                            }
                        }
                    }
                    return __any_sync(kFull, most.over());
                };
                if (form()) {
                    // Scales with which a P' passes the limit are set anew.  A row's largest p s
                    // of each group over the lanes that hold its tokens: values are handed out
                    // while they are compared, so that a lane ends with an eighth of them.
                    constexpr int NV = NCS * RL * NG, NE = NV < 8 ? 1 : NV / 8;
                    float y[NV];
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int cs = i / (RL * NG), e = i / NG % RL, j = i % NG;
                        y[i] = fmaxf(sc[cs][2 * e] * kv4_step(p0[j]), sc[cs][2 * e + 1] * kv4_step(p1[j]));
                    }
                    int n = NV;
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        const bool hi = (lane & o) != 0;
                        if (n == 1) {
                            y[0] = fmaxf(y[0], __shfl_xor_sync(kFull, y[0], o));
                        } else {
                            n /= 2;
#pragma unroll
                            for (int i = 0; i < NV / 2; ++i)
                                if (i < n) {
                                    const float r = __shfl_xor_sync(kFull, hi ? y[i] : y[i + n], o);
                                    y[i] = fmaxf(hi ? y[i + n] : y[i], r);
                                }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NE; ++i) y[i] = pow2i(kMostLog2 - 1 - exponent_of(y[i]));
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int cs = i / (RL * NG), e = i / NG % RL, j = i % NG;
                        const int from = i * 2 / NV * 4 + i * 4 / NV % 2 * 8 + (NV < 8 ? 0 : i * 8 / NV % 2 * 16);
                        const float most = __shfl_sync(kFull, y[i % NE], from + t);
                        if (up[cs][e][j] > most) {
                            const float x = most * kSetUp;
                            scale_row<T>(O[cs][j], e, pow2z(exponent_of(x) - exponent_of(up[cs][e][j])));
                            up[cs][e][j] = x;
                        }
                    }
                    form();
                }
#pragma unroll
                for (int j2 = 0; j2 < NG; j2 += 2) {
                    uint32_t w[4];
                    ldsm4t(w, sa + St::kV + chunk_at<D>(r0 + (lane & 15), j2 + (lane >> 4)));
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        const int j = j2 + jj;
                        const uint32_t wa = w[2 * jj], wb = w[2 * jj + 1];
                        // dims 4g + k of the group, tokens 2t, 2t + 1 (wa) and + 8 (wb)
                        const uint32_t a0 = ctr.low(wa);
                        const uint32_t a1 = ctr.high(wa);
                        const uint32_t a2 = ctr.low(wb);
                        const uint32_t a3 = ctr.high(wb);
                        const uint32_t a4 = ctr.low(wa >> 8);
                        const uint32_t a5 = ctr.high(wa >> 8);
                        const uint32_t a6 = ctr.low(wb >> 8);
                        const uint32_t a7 = ctr.high(wb >> 8);
                        float c0 = fmaf(8.0f, kv4_step(p0[j]), kv4_off(p0[j]));
                        float c1 = fmaf(8.0f, kv4_step(p1[j]), kv4_off(p1[j]));
                        if (CHUNK) {
                            // a NaN group must not reach rows that do not see its token
                            if (c0 != c0) { c0 = 0.0f; nan0 |= 1u << j; }
                            if (c1 != c1) { c1 = 0.0f; nan1 |= 1u << j; }
                        }
#pragma unroll
                        for (int cs = 0; cs < NCS; ++cs) {
#pragma unroll
                            for (int e = 0; e < RL; ++e)
                                bias[cs][e][j] = fmaf(sc[cs][2 * e], c0,
                                                      fmaf(sc[cs][2 * e + 1], c1, bias[cs][e][j]));
                            const uint32_t x0 = movm(b0[cs][j]), x1 = movm(b1[cs][j]);
                            float acc[2][4];
                            mma16816_0(acc[0], a0, a1, a2, a3, x0, x1);
                            mma16816_0(acc[1], a4, a5, a6, a7, x0, x1);
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                O[cs][j][0][z] += acc[0][z];
                                O[cs][j][1][z] += acc[1][z];
                            }
                        }
                    }
                }
                if (CHUNK && (nan0 | nan1)) {
#pragma unroll
                    for (int cs = 0; cs < NCS; ++cs)
#pragma unroll
                        for (int e = 0; e < RL; ++e)
#pragma unroll
                            for (int j = 0; j < NG; ++j)
                                if ((((nan0 >> j) & 1u) && pos0 <= lim[cs][e]) ||
                                    (((nan1 >> j) & 1u) && pos1 <= lim[cs][e]))
                                    bias[cs][e][j] = NAN;
                }
            }
            __syncwarp();
            if (lane == 0 && it + kStagesKv4 < mine)
                fetch(tile0 + warp + (it + kStagesKv4) * kAttendWarps, s);
        }
        if (!alive) {
            // a copy never came: let what is in flight land before the stages are reused
            for (int s = 0; s < kStagesKv4; ++s)
                if (lane == 0) mbar_wait_bounded(&bars[warp][s], (phase >> s) & 1u, c.status, kWaitPollsAfterFail);
        }

        // ---- the warps' results of the unit meet in shared memory (over the ring) ----
        __syncthreads();
        float* red = reinterpret_cast<float*>(ring);   // [warp][RB][D]
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs)
#pragma unroll
            for (int e = 0; e < RL; ++e) {
                const int r = cs * RS + t * RL + e;
                float ls = l[cs][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) ls += __shfl_xor_sync(kFull, ls, o);
                if (g == 0) {
                    red_m[warp][r] = m[cs][e];
                    red_l[warp][r] = ls;
                }
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    float bs = bias[cs][e][j];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) bs += __shfl_xor_sync(kFull, bs, o);
                    float4 v;
                    if constexpr (T == 1) {
                        v.x = O[cs][j][0][e];
                        v.y = O[cs][j][0][2 + e];
                        v.z = O[cs][j][1][e];
                        v.w = O[cs][j][1][2 + e];
                    } else {
                        v.x = fmaf(O[cs][j][0][1], 1.0f / kLowUp, O[cs][j][0][0]);
                        v.y = fmaf(O[cs][j][0][3], 1.0f / kLowUp, O[cs][j][0][2]);
                        v.z = fmaf(O[cs][j][1][1], 1.0f / kLowUp, O[cs][j][1][0]);
                        v.w = fmaf(O[cs][j][1][3], 1.0f / kLowUp, O[cs][j][1][2]);
                    }
                    const float down = pow2i(-exponent_of(up[cs][e][j]));
                    v.x = fmaf(v.x, down, bs);
                    v.y = fmaf(v.y, down, bs);
                    v.z = fmaf(v.z, down, bs);
                    v.w = fmaf(v.w, down, bs);
                    *reinterpret_cast<float4*>(red + ((size_t)warp * RB + r) * D + j * 32 + g * 4) = v;
                }
            }
        __syncthreads();
        const int64_t unit0 = at - tile0;              // first tile of the unit in the list
        const int64_t cta0 = unit0 / quota, cta1 = (unit0 + tiles - 1) / quota;
        const bool whole = cta0 == cta1;
        auto store_row = [&](int r, int d4, float4 v, float mx, float ls) {
            const int row = row0 + r;
            if (row >= row_end || !in_bounds(row < qv.n * c.G && row - row0 < RB, c.status)) return;
            const float inv = ls > 0.0f || ls != ls ? 1.0f / ls : 0.0f;
            const int i = row / c.G, gg = row % c.G;
            TI* o = reinterpret_cast<TI*>(qv.out) +
                    (((int64_t)b * qv.n + i) * c.Hq + h * c.G + gg) * D + d4 * 4;
            if constexpr (T == 2) {
                *reinterpret_cast<float4*>(o) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            } else {
                __nv_bfloat162 y[2] = {__floats2bfloat162_rn(v.x * inv, v.y * inv),
                                       __floats2bfloat162_rn(v.z * inv, v.w * inv)};
                *reinterpret_cast<uint2*>(o) = *reinterpret_cast<uint2*>(y);
            }
            if (d4 == 0) sc_.stat[(int64_t)u * qv.w * c.G + row - qv.i0 * c.G] = kv4_stat(mx, ls);
        };
        auto slot = [&](int64_t cta) {
            if (!in_bounds(cta >= 0 && cta < gridDim.x, c.status)) cta = 0;
            return 2 * cta + (cta == cta0 ? 1 : 0);
        };
        auto part_of = [&](int64_t cta) { return sc_.part + (size_t)slot(cta) * RB * (D + 2); };
        float* part = whole ? nullptr : part_of(blockIdx.x);
        const int nr = row_end - row0 < RB ? row_end - row0 : RB;   // rows of the block that are there
        for (int i = threadIdx.x; i < nr * (D / 4); i += kAttendThreads) {
            const int r = i / (D / 4), d4 = i % (D / 4);
            float mx = red_m[0][r];
#pragma unroll
            for (int w = 1; w < kAttendWarps; ++w) mx = fmaxf(mx, red_m[w][r]);
            float ls = 0.0f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kAttendWarps; ++w) {
                const float f = ex2(red_m[w][r] - mx);
                const float4 x = *reinterpret_cast<const float4*>(red + ((size_t)w * RB + r) * D + d4 * 4);
                ls = fmaf(f, red_l[w][r], ls);
                v.x = fmaf(f, x.x, v.x);
                v.y = fmaf(f, x.y, v.y);
                v.z = fmaf(f, x.z, v.z);
                v.w = fmaf(f, x.w, v.w);
            }
            if (whole) {
                store_row(r, d4, v, mx, ls);
            } else {
                *reinterpret_cast<float4*>(part + r * D + d4 * 4) = v;
                if (d4 == 0) {
                    part[RB * D + r] = mx;
                    part[RB * D + RB + r] = ls;
                }
            }
        }
        if (!whole) {
            // Joined in groups of kJoin CTAs, each by the last of its CTAs to arrive; then
            // the groups' results likewise.  Either way the sums follow the CTAs' order.
            float* fac = reinterpret_cast<float*>(ring);   // [n][RB], over the warps' results
            auto last_of = [&](uint32_t* counter, uint32_t n) {
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0) {
                    last_flag = atomicAdd(counter, 1u) == n - 1;
                    if (last_flag) *counter = 0;
                    __threadfence();
                }
                __syncthreads();
                return last_flag != 0;
            };
            // partials of CTAs first, first + step, ..: into the first's slot, or stored
            auto join = [&](int64_t first, int64_t step, int n, bool store) {
                for (int i = threadIdx.x; i < n * RB; i += kAttendThreads) {
                    const float* p = part_of(first + (i / RB) * step) + RB * D + i % RB;
                    fac[i] = __ldcg(p);
                    fac[n * RB + i] = __ldcg(p + RB);
                }
                __syncthreads();
                if (threadIdx.x < RB) {
                    const int r = threadIdx.x;
                    float mx = kKv4MinLog2, ls = 0.0f;
                    for (int k = 0; k < n; ++k) mx = fmaxf(mx, fac[k * RB + r]);
                    for (int k = 0; k < n; ++k) {
                        const float f = ex2(fac[k * RB + r] - mx);
                        ls = fmaf(f, fac[n * RB + k * RB + r], ls);
                        fac[k * RB + r] = f;
                    }
                    red_m[0][r] = mx;
                    red_l[0][r] = ls;
                }
                __syncthreads();
                float* to = part_of(first);
                for (int i = threadIdx.x; i < nr * (D / 4); i += kAttendThreads) {
                    const int r = i / (D / 4), d4 = i % (D / 4);
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int k = 0; k < n; ++k) {
                        const float f = fac[k * RB + r];
                        const float4 x = __ldcg(reinterpret_cast<const float4*>(
                            part_of(first + k * step) + r * D + d4 * 4));
                        v.x = fmaf(f, x.x, v.x);
                        v.y = fmaf(f, x.y, v.y);
                        v.z = fmaf(f, x.z, v.z);
                        v.w = fmaf(f, x.w, v.w);
                    }
                    if (store) {
                        store_row(r, d4, v, red_m[0][r], red_l[0][r]);
                    } else {
                        *reinterpret_cast<float4*>(to + r * D + d4 * 4) = v;
                        if (d4 == 0) {
                            to[RB * D + r] = red_m[0][r];
                            to[RB * D + RB + r] = red_l[0][r];
                        }
                    }
                }
            };
            const int n = (int)(cta1 - cta0) + 1, groups = (n + kJoin - 1) / kJoin;
            const int64_t first = cta0 + ((int64_t)blockIdx.x - cta0) / kJoin * kJoin;
            const int members = (int)(cta1 - first) + 1 < kJoin ? (int)(cta1 - first) + 1 : kJoin;
            if (last_of(sc_.ucnt + slot(first), members)) {
                join(first, 1, members, groups == 1);
                if (groups > 1 && last_of(sc_.ucnt + 2 * kGridMax + cta0, groups))
                    join(cta0, kJoin, groups, true);
            }
        }
        at += tile1 - tile0;
        // the next unit's copies overwrite what was just read and written here
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
    }
}

// Accumulated weights: w[slot] += sum over the newest acc_rows rows of every sequence
// (all G heads) of 2^(score - m) / l, with the scores formed again from the keys as above (the
// same bits) and the rows' m and l from the attention launch before it.  The difference comes
// first, so that neither large scores nor the logarithm of l cost bits.  The rows that count
// are held in shared memory, as many as fit a launch; a tile's codes are read once for all of
// them.  Every slot belongs to one warp (or one CTA), so sums have one order.
//
// The chunk kernel's own m and l come from keys rounded to fp16; with them a row's weights
// would not add up to 1 (2e-6 off for scores of about 10, a factor for scores of thousands).
// There a launch with SUMS goes first, which forms m and l from these scores.  Units that lie
// whole in a CTA leave them in stat, units that are cut leave a part a CTA: at most one such
// unit begins in a CTA (its last) and one has begun before it, which is two slots a CTA.
//
// Registers: fp32 rows take 168 (three CTAs an SM); held to 128, 16 x 3999 took 3 us more.
//
// Measured: 37 us for one row of 131072 tokens x 8 KV heads (84 MB of keys, 8 of weights); 128
// rows a KV head of 16384 x 8: 115 us for the sums and 86 us for the weights, bound by the
// latency of scores and exponentials at eight warps an SM.
template <int D, int T, bool CHUNK, bool SUMS>
__global__ void __launch_bounds__(kAttendThreads, T == 2 ? 3 : 4) kv4_weights_kernel(
    Kv4View c, Kv4Query qv, Kv4Scratch sc_, const __grid_constant__ Kv4Maps maps, int first_row,
    int n_blocks, int formed) {
    constexpr int NG = D / kKv4Group, RB = 8 / T, RL = 2 / T;
    using St = Stage<D>;
    using RowsT = Rows<D, T, 1>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* ring = smem;
    RowsT* rs = reinterpret_cast<RowsT*>(smem + kAttendWarps * kStagesKv4 * St::kBytes);
    // the rows' m and 1 / l [n_blocks][RB]; SUMS: each warp's m and l [warp][n_blocks][RB]
    float2* stat = reinterpret_cast<float2*>(rs + n_blocks);
    __shared__ Plan pl;
    __shared__ uint64_t bars[kAttendWarps][kStagesKv4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (threadIdx.x == 0) {
        for (int w = 0; w < kAttendWarps; ++w)
            for (int s = 0; s < kStagesKv4; ++s) mbar_init(&bars[w][s], 1);
        mbar_fence_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) make_plan(pl, c, qv, RB, true, CHUNK, lane);
    __syncthreads();
    const int64_t total = pl.pre[c.B];
    int64_t quota = (total + gridDim.x - 1) / gridDim.x;
    // few tiles: a CTA's warps share a tile's blocks of rows instead of taking a tile each
    const bool spread = n_blocks >= kAttendWarps && quota <= 2;
    if (!spread && quota < kAttendWarps) quota = kAttendWarps;
    const int step = spread ? 1 : kAttendWarps, base = spread ? 0 : warp;
    const int k_step = spread ? kAttendWarps : 1, k_base = spread ? warp : 0;
    __shared__ float sums[kAttendWarps][kTile];
    int64_t at = blockIdx.x * quota;
    const int64_t at_end = at + quota < total ? at + quota : total;
    uint32_t phase = 0;
    bool alive = true;
    unsigned char* my_ring = ring + warp * kStagesKv4 * St::kBytes;
    const Centre ctr;
    int b = 0;
    while (at < at_end) {
        while (pl.pre[b + 1] <= at) ++b;
        const int tiles = pl.tiles[b];
        const int64_t in_b = at - pl.pre[b];
        const int h = (int)(in_b / tiles);
        const int tile0 = (int)(in_b - (int64_t)h * tiles);
        const int tile1 = (int)(at_end - at < tiles - tile0 ? at_end - at + tile0 : tiles);
        const int u = b * c.Hkv + h;
        const int64_t L = c.len[b];
        const int n_b = qv.counts ? qv.counts[b] : qv.n;
        // the rows that count: the newest acc_rows of the sequence, within this wave
        int i_lo = n_b - qv.acc_rows > qv.i0 ? n_b - qv.acc_rows : qv.i0;
        const int i_hi = qv.i0 + qv.w < n_b ? qv.i0 + qv.w : n_b;
        const int row0 = i_lo * c.G + first_row;
        const int row_end = i_hi * c.G;
        auto fetch = [&](int tile, int s) {
            unsigned char* st = my_ring + s * St::kBytes;
            uint64_t* bar = &bars[warp][s];
            int64_t r = (int64_t)tile * kTile;
            if (!in_bounds(r >= 0 && r + kTile <= c.R, c.status)) r = 0;
            mbar_expect_tx(bar, St::kCodes + St::kPars + ((CHUNK ? 1 : 0) + (SUMS ? 0 : 1)) * kTile * 4);
            tma_rows(st + St::kK, &maps.k, (int)r, u, bar);
            if (!SUMS) bulk_g2s(st + St::kW, c.w + u * c.R + r, kTile * 4, bar);
            bulk_g2s(st + St::kKp, c.kp + (u * c.R + r) * NG, St::kPars, bar);
            if (CHUNK) bulk_g2s(st + St::kPos, c.pos + u * c.R + r, kTile * 4, bar);
        };
        const int64_t unit0 = at - tile0;              // first tile of the unit in the list
        const int64_t cta0 = unit0 / quota, cta1 = (unit0 + tiles - 1) / quota;
        auto cut_stat = [&](int64_t cta) {
            if (!in_bounds(cta >= 0 && cta < gridDim.x, c.status)) cta = 0;
            return reinterpret_cast<float2*>(sc_.part) + (2 * cta + (cta == cta0 ? 1 : 0)) * n_blocks * RB;
        };
        int mine = L > 0 && row0 < row_end ? (tile1 - tile0 - base + step - 1) / step : 0;
        if (lane == 0 && alive)
            for (int s = 0; s < kStagesKv4 && s < mine; ++s) fetch(tile0 + base + s * step, s);
        const int left = (row_end - row0 + RB - 1) / RB, live_blocks = left < n_blocks ? left : n_blocks;
        if (row0 < row_end) {
            stage_rows<D, T, 1>(rs, n_blocks, c, qv, b, h, row0, row_end, n_b, c.seen[b], warp,
                                kAttendWarps, lane);
            if constexpr (SUMS) {
                for (int i = threadIdx.x; i < kAttendWarps * n_blocks * RB; i += kAttendThreads)
                    stat[i] = make_float2(kKv4MinLog2, 0.0f);
            } else {
                for (int i = threadIdx.x; i < n_blocks * RB; i += kAttendThreads) {
                    float2 x = make_float2(0.0f, 0.0f);
                    if (row0 + i < row_end && !(formed && cta0 != cta1)) {
                        x = sc_.stat[(int64_t)u * qv.w * c.G + row0 + i - qv.i0 * c.G];
                    } else if (row0 + i < row_end) {
                        // (in the order of the CTAs, with a running maximum)
                        float m = kKv4MinLog2, l = 0.0f;
#pragma unroll 4
                        for (int64_t k = cta0; k <= cta1; ++k) {
                            const float2 p = __ldcg(cut_stat(k) + i);
                            const float mn = fmaxf(m, p.x);
                            l = fmaf(p.y, ex2(p.x - mn), l * ex2(m - mn));
                            m = mn;
                        }
                        x = kv4_stat(m, l);
                    }
                    stat[i] = x;
                }
            }
        }
        __syncthreads();
        for (int it = 0; it < mine; ++it) {
            const int s = it % kStagesKv4;
            const int tile = tile0 + base + it * step;
            if (alive && __all_sync(kFull, mbar_wait_bounded(&bars[warp][s], (phase >> s) & 1u, c.status)))
                phase ^= 1u << s;
            else
                alive = false;
            if (!alive && !spread) break;      // (warps that share a tile meet below)
            const unsigned char* st = my_ring + s * St::kBytes;
            const uint32_t sa = smem_u32(st);
#pragma unroll 1
            for (int half = 0; half < 2 && alive; ++half) {
                const int r0 = half * 16;
                const int64_t tok = (int64_t)tile * kTile + r0 + g;
                if (tok - g >= L) break;
                int pos0 = -1, pos1 = -1;
                if (CHUNK) {
                    pos0 = *reinterpret_cast<const int*>(st + St::kPos + (r0 + g) * 4);
                    pos1 = *reinterpret_cast<const int*>(st + St::kPos + (r0 + g + 8) * 4);
                }
                float sum0 = 0.0f, sum1 = 0.0f;
                // several blocks side by side: one alone is a chain of latencies
#pragma unroll 4
                for (int k = k_base; k < live_blocks; k += k_step) {
                    uint4 qreg[NG];
                    float qsum[RL][NG];
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        qreg[j] = rs[k].frag[0][j][lane];
#pragma unroll
                        for (int e = 0; e < RL; ++e) qsum[e][j] = T == 2 ? rs[k].sum[t * RL + e][j] : 0.0f;
                    }
                    float sc[1][2 * RL];
                    scores16<D, T, 1>(sc, st, rs[k], qreg, qsum, rs[k].off[lane], ctr, r0, lane);
#pragma unroll
                    for (int e = 0; e < RL; ++e) {
                        const float f = rs[k].scale[t * RL + e];
                        const int lm = rs[k].lim[t * RL + e];
                        float x0 = __fmul_rn(sc[0][2 * e], f), x1 = __fmul_rn(sc[0][2 * e + 1], f);
                        // rows that are not there have lm = -1, below every position
                        if constexpr (SUMS) {
                            if (!(pos0 <= lm && tok < L)) x0 = -INFINITY;
                            if (!(pos1 <= lm && tok + 8 < L)) x1 = -INFINITY;
                            float2& ml = stat[(warp * n_blocks + k) * RB + t * RL + e];
                            float m = ml.x, l = ml.y, x = fmaxf(x0, x1);
                            if (__any_sync(kFull, x > m + kSlack)) {
                                x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
                                x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
                                x = fmaxf(m, fmaxf(x, __shfl_xor_sync(kFull, x, 16)));
                                l *= ex2(m - x);
                                m = x;
                            }
                            x = ex2(x0 - m) + ex2(x1 - m);
                            x += __shfl_xor_sync(kFull, x, 4);
                            x += __shfl_xor_sync(kFull, x, 8);
                            x += __shfl_xor_sync(kFull, x, 16);
                            if (g == 0) ml = make_float2(m, l + x);
                        } else {
                            const float2 ml = stat[k * RB + t * RL + e];
                            x0 = ex2(x0 - ml.x) * ml.y;
                            x1 = ex2(x1 - ml.x) * ml.y;
                            if ((CHUNK ? pos0 : 0) <= lm) sum0 += x0;
                            if ((CHUNK ? pos1 : 0) <= lm) sum1 += x1;
                        }
                    }
                }
                __syncwarp();                      // (stat is read again by the whole warp)
                if constexpr (SUMS) continue;
                sum0 += __shfl_xor_sync(kFull, sum0, 1);
                sum1 += __shfl_xor_sync(kFull, sum1, 1);
                sum0 += __shfl_xor_sync(kFull, sum0, 2);
                sum1 += __shfl_xor_sync(kFull, sum1, 2);
                if (t == 0 && spread) {
                    sums[warp][r0 + g] = sum0;
                    sums[warp][r0 + g + 8] = sum1;
                } else if (t == 0) {
                    // this warp's alone: what the tile brought, and more
                    const float* old = reinterpret_cast<const float*>(st + St::kW) + r0 + g;
                    float* w = c.w + u * c.R + tok;
                    if (tok < L && in_bounds(tok < c.cap, c.status)) w[0] = old[0] + sum0;
                    if (tok + 8 < L && in_bounds(tok + 8 < c.cap, c.status)) w[8] = old[8] + sum1;
                }
            }
            if (spread && !SUMS) {
                __syncthreads();
                const int64_t tok = (int64_t)tile * kTile + lane;
                if (warp == 0 && alive && tok < L && in_bounds(tok < c.cap, c.status)) {
                    float x = reinterpret_cast<const float*>(st + St::kW)[lane];
#pragma unroll
                    for (int i = 0; i < kAttendWarps; ++i) x += sums[i][lane];
                    c.w[u * c.R + tok] = x;
                }
                __syncthreads();
            }
            __syncwarp();
            if (lane == 0 && alive && it + kStagesKv4 < mine)
                fetch(tile0 + base + (it + kStagesKv4) * step, s);
        }
        if (!alive) {
            for (int s = 0; s < kStagesKv4; ++s)
                if (lane == 0) mbar_wait_bounded(&bars[warp][s], (phase >> s) & 1u, c.status, kWaitPollsAfterFail);
        }
        if constexpr (SUMS) {
            __syncthreads();
            for (int i = threadIdx.x; row0 + i < row_end && i < n_blocks * RB; i += kAttendThreads) {
                float m = kKv4MinLog2, l = 0.0f;
#pragma unroll
                for (int k = 0; k < kAttendWarps; ++k) m = fmaxf(m, stat[k * n_blocks * RB + i].x);
#pragma unroll
                for (int k = 0; k < kAttendWarps; ++k) {
                    const float2 p = stat[k * n_blocks * RB + i];
                    l = fmaf(p.y, ex2(p.x - m), l);
                }
                if (!in_bounds(row0 + i - qv.i0 * c.G < qv.w * c.G, c.status)) continue;
                if (cta0 == cta1)
                    sc_.stat[(int64_t)u * qv.w * c.G + row0 + i - qv.i0 * c.G] = kv4_stat(m, l);
                else
                    cut_stat(blockIdx.x)[i] = make_float2(m, l);
            }
        }
        at += tile1 - tile0;
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------------
namespace {

template <int D, int T, int NCS>
constexpr size_t attend_smem() {
    return 1024 + ring_bytes<D, NCS * 8 / T>() + sizeof(Rows<D, T, NCS>);
}
// A column set's rows and their statistics (bf16: each warp's, for SUMS).
template <int D, int T>
constexpr size_t weights_block_bytes() {
    return sizeof(Rows<D, T, 1>) + (T == 1 ? kAttendWarps : 1) * sizeof(float2) * 8 / T;
}
template <int D, int T>
constexpr size_t weights_smem(int blocks) {
    return 1024 + (size_t)kAttendWarps * kStagesKv4 * Stage<D>::kBytes +
           (size_t)blocks * weights_block_bytes<D, T>();
}
// Column sets a weights launch holds: 64 KB of rows, so that two CTAs share an SM beside
// their rings (four with half of it).
template <int D, int T>
constexpr int weight_blocks() {
    return 65536 / (int)weights_block_bytes<D, T>();
}

// Column sets of a block: the fewest that hold the rows, up to four (the accumulators of
// four fill the register file).
int sets_for(int T, int rows) {
    const int per = 8 / T;
    return rows <= per ? 1 : rows <= 2 * per ? 2 : 4;
}

template <typename K>
cudaError_t allow(K kern, size_t smem) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

template <int D, int T>
cudaError_t prepare_impl() {
    cudaError_t e = allow(kv4_attend_kernel<D, T, 1, false>, attend_smem<D, T, 1>());
    if constexpr (T == 2)
        if (e == cudaSuccess) e = allow(kv4_attend_kernel<D, T, 2, false>, attend_smem<D, T, 2>());
    if (e == cudaSuccess) e = allow(kv4_attend_kernel<D, T, 1, true>, attend_smem<D, T, 1>());
    if constexpr (T == 2) {
        if (e == cudaSuccess) e = allow(kv4_attend_kernel<D, T, 2, true>, attend_smem<D, T, 2>());
        if (e == cudaSuccess) e = allow(kv4_attend_kernel<D, T, 4, true>, attend_smem<D, T, 4>());
    }
    const size_t most = weights_smem<D, T>(weight_blocks<D, T>());
    if (e == cudaSuccess) e = allow(kv4_weights_kernel<D, T, false, false>, most);
    if (e == cudaSuccess) e = allow(kv4_weights_kernel<D, T, true, false>, most);
    if constexpr (T == 1)
        if (e == cudaSuccess) e = allow(kv4_weights_kernel<D, T, true, true>, most);
    return e;
}

template <int D, int T>
cudaError_t attend_impl(const Kv4View& c, const Kv4Query& qv, const Kv4Scratch& sc,
                        const Kv4Maps& maps, int chunk, cudaStream_t s) {
    const int sets = sets_for(T, qv.w * c.G);
    const dim3 grid(148 * (sets == 1 ? ctas_per_sm<1>() : sets == 2 ? ctas_per_sm<2>()
                                                                     : ctas_per_sm<4>()));
    if (!chunk) {
        if (sets == 1)
            return kv4_launch(kv4_attend_kernel<D, T, 1, false>, grid, kAttendThreads,
                              attend_smem<D, T, 1>(), s, c, qv, sc, maps);
        if constexpr (T == 2)
            return kv4_launch(kv4_attend_kernel<D, T, 2, false>, grid, kAttendThreads,
                              attend_smem<D, T, 2>(), s, c, qv, sc, maps);
        return cudaErrorInvalidValue;   // bf16: 8 columns hold the 8 heads of the largest group
    }
    if (sets == 1)
        return kv4_launch(kv4_attend_kernel<D, T, 1, true>, grid, kAttendThreads,
                          attend_smem<D, T, 1>(), s, c, qv, sc, maps);
    if constexpr (T == 2) {
        if (sets == 2)
            return kv4_launch(kv4_attend_kernel<D, T, 2, true>, grid, kAttendThreads,
                              attend_smem<D, T, 2>(), s, c, qv, sc, maps);
        return kv4_launch(kv4_attend_kernel<D, T, 4, true>, grid, kAttendThreads,
                          attend_smem<D, T, 4>(), s, c, qv, sc, maps);
    }
    return cudaErrorInvalidValue;   // more bf16 rows are the chunk kernel's
}

template <int D, int T>
cudaError_t weights_impl(const Kv4View& c, const Kv4Query& qv, const Kv4Scratch& sc,
                         const Kv4Maps& maps, int chunk, int form_stat, cudaStream_t s) {
    const int rows = (qv.acc_rows < qv.w ? qv.acc_rows : qv.w) * c.G, per = 8 / T;
    constexpr int most = weight_blocks<D, T>();
    // two slots of (m, l) a CTA for the units that are cut
    static_assert(T == 2 || 2 * most * 8 * 2 <= 2 * 16 * (D + 2), "the parts do not hold them");
    for (int r = 0; r < rows; r += most * per) {
        int blocks = (rows - r + per - 1) / per;
        if (blocks > most) blocks = most;
        const size_t smem = weights_smem<D, T>(blocks);
        const dim3 grid(148 * (smem <= 56 * 1024 ? 4 : smem <= 74 * 1024 ? 3 : 2));
        cudaError_t e = cudaSuccess;
        if constexpr (T == 1)
            if (form_stat)
                e = kv4_launch(kv4_weights_kernel<D, T, true, true>, grid, kAttendThreads, smem, s, c, qv,
                               sc, maps, r, blocks, 0);
        if (e != cudaSuccess) return e;
        e = chunk ? kv4_launch(kv4_weights_kernel<D, T, true, false>, grid, kAttendThreads, smem, s, c, qv,
                               sc, maps, r, blocks, form_stat)
                  : kv4_launch(kv4_weights_kernel<D, T, false, false>, grid, kAttendThreads, smem, s, c,
                               qv, sc, maps, r, blocks, 0);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

int kv4_attend_counters() { return 3 * kGridMax; }
size_t kv4_attend_part_floats(int D) { return (size_t)2 * kGridMax * 16 * (D + 2); }

#define KV4_ATTEND(FN, ...)                                             \
    do {                                                                \
        if (dtype == RECSA_BF16 && D_ == 128) return FN<128, 1>(__VA_ARGS__); \
        if (dtype == RECSA_BF16 && D_ == 64) return FN<64, 1>(__VA_ARGS__);   \
        if (dtype == RECSA_F32 && D_ == 128) return FN<128, 2>(__VA_ARGS__);  \
        if (dtype == RECSA_F32 && D_ == 64) return FN<64, 2>(__VA_ARGS__);    \
        return cudaErrorInvalidValue;                                   \
    } while (0)

cudaError_t kv4_prepare_attend(int dtype, int D_) { KV4_ATTEND(prepare_impl); }

cudaError_t kv4_launch_attend(const Kv4View& c, const Kv4Query& qv, const Kv4Scratch& sc,
                              const Kv4Maps& maps, int chunk, int dtype, cudaStream_t s) {
    NvtxRange nv("recsa kv4 attend");
    const int D_ = c.D;
    KV4_ATTEND(attend_impl, c, qv, sc, maps, chunk, s);
}

cudaError_t kv4_launch_weights(const Kv4View& c, const Kv4Query& qv, const Kv4Scratch& sc,
                               const Kv4Maps& maps, int chunk, int form_stat, int dtype, cudaStream_t s) {
    NvtxRange nv("recsa kv4 weights");
    const int D_ = c.D;
    KV4_ATTEND(weights_impl, c, qv, sc, maps, chunk, form_stat, s);
}

}  // namespace recsa
