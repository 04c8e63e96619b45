// Host side of the 4-bit KV cache (recsa_kv4_*): argument checks, buffer layout, launches.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include <mutex>

#include "kv4.cuh"

namespace recsa {

namespace {

constexpr int64_t kMaxCapacity = (int64_t)1 << 30;   // rows: slots and positions are int32

struct Kv4Layout {
    int D, G, esize;
    int64_t R, U;
    size_t o_kc, o_vc, o_kp, o_vp, o_pos, o_w, cache_bytes;
    size_t o_status, o_done, o_len, o_seen, o_kmax, o_vmax, o_kmin, o_vmin, o_wide, o_ucnt, o_stat, o_part, o_sum, o_lists, ws_bytes;
};

// Rows (chunk rows times heads of a group) of one wave and KV head that kv4_launch_chunk takes:
// what does not fit the 8 columns of the other kernel's narrowest form, in bf16.  Chunk kernel /
// the other with a block for every 8 rows, us, 8 KV heads, d = 128:
//     sequences x tokens   12 rows    16         20         32         64
//     1 x 1500             23/25      25/27      26/26      27/29      29/28
//     1 x 9000             46/33      47/34      48/36      50/42      53/49
//     8 x 9000             85/78      87/78      92/104     94/131     94/236
//     1 x 131072           142/123    141/124    148/171    145/218    148/407
//     4 x 131072           403/407    407/408    409/598    410/789    412/1548
bool chunk_on_tensor_cores(int dtype, int rows) { return dtype == RECSA_BF16 && rows > 8; }

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
// May a call read its queries from q and write its rows to out, `bytes` each?  In place, yes,
// unless a second launch reads the queries again (for weights); a partial overlap, never.
bool apart(const void* q, const void* out, size_t bytes, bool again) {
    const uintptr_t a = (uintptr_t)q, b = (uintptr_t)out;
    if (a == b) return !again;
    return a < b ? b - a >= bytes : a - b >= bytes;
}
bool on16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

recsa_status kv4_layout(const recsa_config* c, int64_t cap, int B, int Qmax, Kv4Layout* L) {
    if (!c) return RECSA_E_INVAL;
    if (c->n_q_heads <= 0 || c->n_kv_heads <= 0 || c->n_q_heads % c->n_kv_heads) return RECSA_E_INVAL;
    if (c->dtype != RECSA_F32 && c->dtype != RECSA_BF16) return RECSA_E_INVAL;
    if (!(c->scale >= 0.0f) || !isfinite(c->scale)) return RECSA_E_INVAL;
    if (c->head_dim != 64 && c->head_dim != 128) return RECSA_E_UNSUPPORTED;
    const int G = c->n_q_heads / c->n_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return RECSA_E_UNSUPPORTED;
    if (cap < 1 || B < 1 || B > RECSA_MAX_BATCH || Qmax < B || Qmax > (1 << 20)) return RECSA_E_INVAL;
    if (cap > kMaxCapacity || (int64_t)B * c->n_kv_heads > 65535) return RECSA_E_UNSUPPORTED;
    memset(L, 0, sizeof(*L));
    L->D = c->head_dim;
    L->G = G;
    L->esize = c->dtype == RECSA_BF16 ? 2 : 4;
    L->R = (cap + kKv4RowPad - 1) / kKv4RowPad * kKv4RowPad;
    L->U = (int64_t)B * c->n_kv_heads;
    const size_t rows = (size_t)L->U * (size_t)L->R;
    size_t o = 0;
    L->o_kc = o;  o = up256(o + rows * L->D / 2);
    L->o_vc = o;  o = up256(o + rows * L->D / 2);
    L->o_kp = o;  o = up256(o + rows * L->D / 8);
    L->o_vp = o;  o = up256(o + rows * L->D / 8);
    L->o_pos = o; o = up256(o + rows * 4);
    L->o_w = o;   o = up256(o + rows * 4);
    L->cache_bytes = o;
    size_t w = 0;
    L->o_status = w; w = up256(w + 64);
    L->o_done = w;   w = up256(w + 64);
    L->o_len = w;    w = up256(w + sizeof(int64_t) * B);
    L->o_seen = w;   w = up256(w + sizeof(int64_t) * B);
    L->o_kmax = w;   w = up256(w + sizeof(uint32_t) * L->U);
    L->o_vmax = w;   w = up256(w + sizeof(uint32_t) * L->U);
    L->o_kmin = w;   w = up256(w + sizeof(uint32_t) * L->U);
    L->o_vmin = w;   w = up256(w + sizeof(uint32_t) * L->U);
    L->o_wide = w;   w = up256(w + sizeof(uint32_t) * B);
    L->o_ucnt = w;   w = up256(w + sizeof(uint32_t) * kv4_attend_counters());
    L->o_stat = w;   w = up256(w + sizeof(float2) * (size_t)Qmax * c->n_q_heads);
    size_t part = kv4_attend_part_floats(L->D), sum = 0;
    if (chunk_on_tensor_cores(c->dtype, Qmax / B * G)) {
        sum = kv4_chunk_sum_floats(L->D, L->R);
        const size_t p = kv4_chunk_part_floats(L->D, Qmax / B * G);
        if (p > part) part = p;
    }
    L->o_part = w;   w = up256(w + sizeof(float) * part);
    L->o_sum = w;    w = up256(w + sizeof(float) * sum);
    L->o_lists = w;  w = up256(w + sizeof(int32_t) * rows);
    L->ws_bytes = w;
    return RECSA_OK;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);

EncodeFn encode_entry() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

// Codes of one tensor: (bytes of a row, row, unit), boxes of `rows` whole rows, swizzled
// so that eight rows' 16-byte pieces of one group lie in eight different bank groups.
bool encode_codes(CUtensorMap* m, void* base, int D, int64_t R, int64_t U, int rows) {
    EncodeFn fn = encode_entry();
    if (!fn) return false;
    const cuuint64_t row = (cuuint64_t)D / 2;
    const cuuint64_t dims[3] = {row, (cuuint64_t)R, (cuuint64_t)U};
    const cuuint64_t strides[2] = {row, row * (cuuint64_t)R};
    const cuuint32_t box[3] = {(cuuint32_t)row, (cuuint32_t)rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool device_memory(const void* p, int* dev) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    *dev = a.device;
    return a.type == cudaMemoryTypeDevice;
}

}  // namespace

}  // namespace recsa

using namespace recsa;

struct recsa_kv4 {
    recsa_config cfg;
    Kv4Layout L;
    int Qmax, device;
    Kv4View c;
    Kv4Scratch sc;
    Kv4Maps maps;
    int32_t* lists;
};

namespace {

// Makes the cache's device current for a call and puts the caller's back.
struct OnDevice {
    int before = -1;
    bool ok;
    explicit OnDevice(int dev) {
        ok = cudaGetDevice(&before) == cudaSuccess;
        if (ok && before != dev) ok = cudaSetDevice(dev) == cudaSuccess;
        else before = -1;
    }
    ~OnDevice() {
        if (before >= 0) cudaSetDevice(before);
    }
};

recsa_status done(cudaError_t e) { return e == cudaSuccess ? RECSA_OK : RECSA_E_CUDA; }

}  // namespace

extern "C" {

recsa_status recsa_kv4_query_sizes(const recsa_config* cfg, int64_t capacity, int32_t batch,
                                   int32_t max_queries, size_t* cache_bytes,
                                   size_t* workspace_bytes) {
    Kv4Layout L;
    const recsa_status st = kv4_layout(cfg, capacity, batch, max_queries, &L);
    if (st != RECSA_OK) return st;
    if (cache_bytes) *cache_bytes = L.cache_bytes;
    if (workspace_bytes) *workspace_bytes = L.ws_bytes;
    return RECSA_OK;
}

recsa_status recsa_kv4_init(const recsa_config* cfg, int64_t capacity, int32_t batch,
                            int32_t max_queries, void* cache, size_t cache_bytes, void* workspace,
                            size_t workspace_bytes, void* stream, recsa_kv4** out) {
    if (!out) return RECSA_E_INVAL;
    *out = nullptr;
    Kv4Layout L;
    recsa_status st = kv4_layout(cfg, capacity, batch, max_queries, &L);
    if (st != RECSA_OK) return st;
    if (!cache || !workspace) return RECSA_E_INVAL;
    if (((uintptr_t)cache & 255u) || ((uintptr_t)workspace & 255u)) return RECSA_E_INVAL;
    if (cache_bytes < L.cache_bytes || workspace_bytes < L.ws_bytes) return RECSA_E_CAPACITY;
    int dev = -1, dev_ws = -1;
    if (!device_memory(cache, &dev) || !device_memory(workspace, &dev_ws) || dev != dev_ws)
        return RECSA_E_INVAL;
    recsa_kv4* t = (recsa_kv4*)calloc(1, sizeof(recsa_kv4));
    if (!t) return RECSA_E_INVAL;
    t->cfg = *cfg;
    t->L = L;
    t->Qmax = max_queries;
    t->device = dev;
    char *cb = (char*)cache, *ws = (char*)workspace;
    Kv4View& c = t->c;
    c.kc = (uint8_t*)(cb + L.o_kc);
    c.vc = (uint8_t*)(cb + L.o_vc);
    c.kp = (uint32_t*)(cb + L.o_kp);
    c.vp = (uint32_t*)(cb + L.o_vp);
    c.pos = (int32_t*)(cb + L.o_pos);
    c.w = (float*)(cb + L.o_w);
    c.status = (uint32_t*)(ws + L.o_status);
    c.done = (uint32_t*)(ws + L.o_done);
    c.len = (int64_t*)(ws + L.o_len);
    c.seen = (int64_t*)(ws + L.o_seen);
    c.kmax = (uint32_t*)(ws + L.o_kmax);
    c.vmax = (uint32_t*)(ws + L.o_vmax);
    c.kmin = (uint32_t*)(ws + L.o_kmin);
    c.vmin = (uint32_t*)(ws + L.o_vmin);
    c.wide = (uint32_t*)(ws + L.o_wide);
    c.B = batch;
    c.Hkv = cfg->n_kv_heads;
    c.Hq = cfg->n_q_heads;
    c.G = L.G;
    c.D = L.D;
    c.R = L.R;
    c.cap = capacity;
    c.scale = cfg->scale > 0.0f ? cfg->scale : (float)(1.0 / sqrt((double)L.D));
    t->sc.ucnt = (uint32_t*)(ws + L.o_ucnt);
    t->sc.stat = (float2*)(ws + L.o_stat);
    t->sc.part = (float*)(ws + L.o_part);
    t->sc.sum = (float4*)(ws + L.o_sum);
    t->lists = (int32_t*)(ws + L.o_lists);
    OnDevice on(dev);
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = on.ok ? kv4_prepare_attend(cfg->dtype, L.D) : cudaErrorInvalidDevice;
    if (e == cudaSuccess) e = kv4_prepare_evict(c);
    if (e == cudaSuccess) e = kv4_prepare_chunk(L.D);
    if (e == cudaSuccess && (!encode_codes(&t->maps.k, c.kc, L.D, L.R, L.U, 32) ||
                             !encode_codes(&t->maps.v, c.vc, L.D, L.R, L.U, 32)))
        e = cudaErrorNotSupported;
    if (e == cudaSuccess)
        e = cudaMemsetAsync(t->sc.ucnt, 0, sizeof(uint32_t) * kv4_attend_counters(), s);
    if (e == cudaSuccess) e = kv4_launch_clear(c, s);
    if (e != cudaSuccess) {
        free(t);
        return RECSA_E_CUDA;
    }
    *out = t;
    return RECSA_OK;
}

recsa_status recsa_kv4_build(recsa_kv4* t, const void* k, const void* v, const int64_t kv_strides[3],
                             const int64_t* lengths, void* stream) {
    if (!t || !k || !v || !kv_strides || !lengths) return RECSA_E_INVAL;
    if (!on16(k) || !on16(v)) return RECSA_E_INVAL;
    const int64_t per16 = 16 / t->L.esize;
    for (int i = 0; i < 3; ++i)
        if (kv_strides[i] < 0 || kv_strides[i] % per16) return RECSA_E_INVAL;
    if (kv_strides[2] < t->L.D) return RECSA_E_INVAL;
    Kv4Lengths lens = {};
    Kv4Source src = {};
    src.n = 1;                           // all empty: one CTA a unit still sets the lengths
    for (int b = 0; b < t->c.B; ++b) {
        if (lengths[b] < 0) return RECSA_E_INVAL;
        if (lengths[b] > t->c.cap) return RECSA_E_CAPACITY;
        lens.v[b] = lengths[b];
        if (lengths[b] > src.n) src.n = lengths[b];
    }
    src.k = k;
    src.v = v;
    src.s_b = kv_strides[0];
    src.s_h = kv_strides[1];
    src.s_t = kv_strides[2];
    OnDevice on(t->device);
    if (!on.ok) return RECSA_E_CUDA;
    return done(kv4_launch_build(t->c, src, lens, t->cfg.dtype, (cudaStream_t)stream));
}

recsa_status recsa_kv4_append(recsa_kv4* t, const void* k_new, const void* v_new, int32_t n,
                              const int32_t* counts, void* stream) {
    if (!t || !k_new || !v_new || n < 1) return RECSA_E_INVAL;
    if (!on16(k_new) || !on16(v_new) || ((uintptr_t)counts & 3u)) return RECSA_E_INVAL;
    if (n > t->c.cap) return RECSA_E_CAPACITY;
    Kv4Source src = {};
    src.k = k_new;
    src.v = v_new;
    src.s_t = t->L.D;
    src.s_h = (int64_t)n * t->L.D;
    src.s_b = src.s_h * t->c.Hkv;
    src.n = n;
    src.counts = counts;
    src.append = 1;
    OnDevice on(t->device);
    if (!on.ok) return RECSA_E_CUDA;
    return done(kv4_launch_append(t->c, src, t->cfg.dtype, (cudaStream_t)stream));
}

recsa_status recsa_kv4_decode(recsa_kv4* t, const void* q, void* out, int32_t accumulate,
                              void* stream) {
    if (!t || !q || !out) return RECSA_E_INVAL;
    if (!on16(q) || !on16(out)) return RECSA_E_INVAL;
    const size_t bytes = (size_t)t->c.B * t->c.Hq * t->L.D * t->L.esize;
    if (!apart(q, out, bytes, accumulate != 0)) return RECSA_E_INVAL;
    Kv4Query qv = {};
    qv.q = q;
    qv.out = out;
    qv.n = qv.w = 1;
    qv.acc_rows = accumulate ? 1 : 0;
    OnDevice on(t->device);
    if (!on.ok) return RECSA_E_CUDA;
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = kv4_launch_attend(t->c, qv, t->sc, t->maps, 0, t->cfg.dtype, s);
    if (e == cudaSuccess && accumulate)
        e = kv4_launch_weights(t->c, qv, t->sc, t->maps, 0, 0, t->cfg.dtype, s);
    return done(e);
}

recsa_status recsa_kv4_prefill_chunk(recsa_kv4* t, const void* Q, int32_t n, const int32_t* counts,
                                     void* O, int32_t accumulate_rows, void* stream) {
    if (!t || !Q || !O || n < 1 || accumulate_rows < 0) return RECSA_E_INVAL;
    if (!on16(Q) || !on16(O) || ((uintptr_t)counts & 3u)) return RECSA_E_INVAL;
    const size_t bytes = (size_t)t->c.B * n * t->c.Hq * t->L.D * t->L.esize;
    if (!apart(Q, O, bytes, accumulate_rows != 0)) return RECSA_E_INVAL;
    OnDevice on(t->device);
    if (!on.ok) return RECSA_E_CUDA;
    const cudaStream_t s = (cudaStream_t)stream;
    const int wave = t->Qmax / t->c.B;   // rows a sequence of one wave
    cudaError_t e = cudaSuccess;
    for (int i0 = 0; i0 < n && e == cudaSuccess; i0 += wave) {
        Kv4Query qv = {};
        qv.q = Q;
        qv.out = O;
        qv.counts = counts;
        qv.n = n;
        qv.i0 = i0;
        qv.w = n - i0 < wave ? n - i0 : wave;
        qv.acc_rows = accumulate_rows < n ? accumulate_rows : n;
        const bool tc = chunk_on_tensor_cores(t->cfg.dtype, qv.w * t->c.G);
        e = tc ? kv4_launch_chunk(t->c, qv, t->sc, s)
               : kv4_launch_attend(t->c, qv, t->sc, t->maps, 1, t->cfg.dtype, s);
        // with counts the newest rows may lie in any wave, else in the last ones
        if (e == cudaSuccess && qv.acc_rows > 0 && (counts || i0 + qv.w > n - qv.acc_rows))
            e = kv4_launch_weights(t->c, qv, t->sc, t->maps, 1, tc, t->cfg.dtype, s);
    }
    return done(e);
}

recsa_status recsa_kv4_evict(recsa_kv4* t, int64_t budget, int64_t n_first, int64_t n_recent,
                             void* stream) {
    if (!t || budget < 1 || n_first < 0 || n_recent < 0) return RECSA_E_INVAL;
    if (n_first > budget || n_recent > budget - n_first) return RECSA_E_INVAL;
    OnDevice on(t->device);
    if (!on.ok) return RECSA_E_CUDA;
    return done(kv4_launch_evict(t->c, budget, n_first, n_recent, t->lists, (cudaStream_t)stream));
}

recsa_status recsa_kv4_read(recsa_kv4* t, int64_t start, int64_t n, void* k_out, void* v_out,
                            void* stream) {
    if (!t || start < 0 || n < 1 || (!k_out && !v_out)) return RECSA_E_INVAL;
    if (!on16(k_out) || !on16(v_out)) return RECSA_E_INVAL;
    if (start > t->c.cap || n > t->c.cap - start) return RECSA_E_CAPACITY;
    OnDevice on(t->device);
    if (!on.ok) return RECSA_E_CUDA;
    return done(kv4_launch_read(t->c, start, n, k_out, v_out, t->cfg.dtype, (cudaStream_t)stream));
}

recsa_status recsa_kv4_get_status(recsa_kv4* t, void* stream) {
    if (!t) return RECSA_E_INVAL;
    OnDevice on(t->device);
    if (!on.ok) return RECSA_E_CUDA;
    const cudaStream_t s = (cudaStream_t)stream;
    uint32_t v = 0;
    if (cudaMemcpyAsync(&v, t->c.status, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return RECSA_E_CUDA;
    if (v != 0 && (cudaMemsetAsync(t->c.status, 0, sizeof(v), s) != cudaSuccess ||
                   cudaStreamSynchronize(s) != cudaSuccess))
        return RECSA_E_CUDA;
    switch (v) {
        case kStatusOk: return RECSA_OK;
        case kStatusCapacity: return RECSA_E_CAPACITY;
        case kStatusTimeout: return RECSA_E_TIMEOUT;
        default: return RECSA_E_DEVICE;
    }
}

recsa_status recsa_kv4_info(const recsa_kv4* t, recsa_kv4_info_t* info) {
    if (!t || !info) return RECSA_E_INVAL;
    info->capacity = t->c.cap;
    info->rows = t->L.R;
    info->batch = t->c.B;
    info->max_queries = t->Qmax;
    info->k_codes = (int64_t)t->L.o_kc;
    info->v_codes = (int64_t)t->L.o_vc;
    info->k_params = (int64_t)t->L.o_kp;
    info->v_params = (int64_t)t->L.o_vp;
    info->positions = (int64_t)t->L.o_pos;
    info->weights = (int64_t)t->L.o_w;
    info->lengths = (int64_t)t->L.o_len;
    info->tokens_seen = (int64_t)t->L.o_seen;
    return RECSA_OK;
}

recsa_status recsa_kv4_free(recsa_kv4* t) {
    if (!t) return RECSA_E_INVAL;
    free(t);
    return RECSA_OK;
}

}  // extern "C"
