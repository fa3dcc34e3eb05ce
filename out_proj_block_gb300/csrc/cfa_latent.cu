// cfa_latent.cu -- host side of the paged latent-cache entry points (include/cfa.h):
// argument checks, the workspace and the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <new>

#include "cfa.h"
#include "cfa_host.h"
#include "cfa_host_util.h"
#include "cfa_internal.h"
#include "cfa_latent.h"
#include "cfa_latent_split.h"
#include "cfa_paged.h"

namespace cfa {
const void *latent_append_kernel_ptr(bool interleaved);
const void *latent_heads_kernel_ptr(bool fold);
int latent_heads_smem(bool fold);
const void *latent_heads_mma_kernel_ptr(bool fold);
int latent_heads_mma_smem(bool fold);
const void *latent_attention_kernel_ptr();
const void *latent_merge_kernel_ptr();
const void *latent_expanded_kernel_ptr();
const void *latent_expanded_merge_kernel_ptr();
int latent_expanded_smem();
int latent_attention_smem();
}  // namespace cfa

struct cfa_latent {
    int max_seqs = 0, max_tokens = 0, nh = 0, ps = 0;
    int device = -1, num_sms = 0;
    // rotation
    int rope = 0, interleaved = 0, scaling = CFA_ROPE_PLAIN;
    float magnitude = 1.0f;
    unsigned long long turns[cfa::kLatR / 2] = {};
    // workspace
    unsigned *words = nullptr;  // kLatWords: [0] status, [1..] the expanded form's merge (odd, rest, odd_tiles)
    float *rec_o = nullptr;     // records of the attention's pieces
    float2 *rec_ml = nullptr;
    int4 *cuts = nullptr;
    int runs = 0;
};

namespace {

using cfa::OnDevice;
using cfa::Span;
using cfa::aligned;
using cfa::clear_words;
using cfa::kLatC;
using cfa::kLatKv;
using cfa::kLatQ;
using cfa::kLatR;
using cfa::kLatRow;
using cfa::kLatV;
using cfa::overlaps;

constexpr uint32_t kTimeoutNs = 2000000000u;  // 2 s per device-side wait

cfa_status fail(cfa_status s) { return cfa::set_last_error(s); }

void latent_free(cfa_latent *p) {
    void *all[] = {p->words, p->rec_o, p->rec_ml, p->cuts};
    for (void *a : all)
        if (a) cudaFree(a);
}

// Rows of a cache of n_pages pages, or -1 where they pass the kernels' 32-bit row index.
long long cache_rows(const cfa_latent *p, int n_pages) {
    return n_pages > ((1ll << 31) - 1) / p->ps ? -1 : static_cast<long long>(n_pages) * p->ps;
}

// Bytes that n rows of `width` elements with this stride span.
size_t span(int n, long long width, long long stride) {
    return n ? 2u * (static_cast<size_t>(n - 1) * static_cast<size_t>(stride) + static_cast<size_t>(width)) : 0;
}

bool stride_ok(long long width, long long stride) {
    return stride >= width && stride % 8 == 0 && stride < (1ll << 36);
}

// Whether what a call writes lies apart from what it reads and from its other results.
bool apart(std::initializer_list<Span> writes, std::initializer_list<Span> reads) {
    for (const Span *w = writes.begin(); w != writes.end(); ++w) {
        for (const Span &r : reads)
            if (overlaps(w->at, w->n, r.at, r.n)) return false;
        for (const Span *v = writes.begin(); v != w; ++v)
            if (overlaps(w->at, w->n, v->at, v->n)) return false;
    }
    return true;
}

bool aligned_to(uintptr_t to, std::initializer_list<const void *> all) {
    for (const void *p : all)
        if (!aligned(p, to)) return false;
    return true;
}

struct AppendArgs {
    int n_tokens;
    const void *a;
    long long as;
    const void *g;
    float eps;
    const void *q;
    long long qs;
    const int *positions, *slots;
    int n_pages;
    void *pages, *q_out;
};

struct AttnArgs {
    int n_tokens, n_seqs;
    const void *q;
    const int *cu, *tables;
    int width;
    const int *lens;
    int n_pages;
    const void *pages;
    float scale;
    void *out;
    float *lse;
};

size_t page_bytes(const cfa_latent *p, int n_pages) { return 2u * static_cast<size_t>(cache_rows(p, n_pages)) * kLatRow; }
size_t weight_bytes(const cfa_latent *p) { return 2u * kLatC * kLatKv * static_cast<size_t>(p->nh); }
// Bytes of [n][n_heads][d] bf16.
size_t heads_bytes(const cfa_latent *p, int n, int d) { return 2u * static_cast<size_t>(n) * p->nh * d; }

bool tokens_ok(const cfa_latent *p, int n) { return n >= 0 && n <= p->max_tokens; }
bool in_place(const cfa_latent *p, const AppendArgs &a) {
    return a.q_out == a.q && a.qs == static_cast<long long>(p->nh) * kLatQ;
}

cfa_status check_append(const cfa_latent *p, const AppendArgs &a) {
    const long long wide = static_cast<long long>(p->nh) * kLatQ;
    if (!a.a || !a.g || !a.q || !a.positions || !a.slots || !a.pages || !a.q_out || a.n_pages < 1 ||
        cache_rows(p, a.n_pages) < 0 || !stride_ok(kLatRow, a.as) || !stride_ok(wide, a.qs) ||
        !(a.eps >= 0.0f) || !std::isfinite(a.eps))
        return CFA_ERR_INVALID_ARG;
    if (!aligned_to(16, {a.a, a.g, a.q, a.pages, a.q_out}) || !aligned_to(4, {a.positions, a.slots}))
        return CFA_ERR_ALIGNMENT;
    const size_t ints = 4u * static_cast<size_t>(a.n_tokens);
    const Span q{a.q, in_place(p, a) ? 0 : span(a.n_tokens, wide, a.qs)};
    return apart({{a.pages, page_bytes(p, a.n_pages)}, {a.q_out, heads_bytes(p, a.n_tokens, kLatQ)}},
                 {{a.a, span(a.n_tokens, kLatRow, a.as)}, {a.g, 2 * kLatC}, q, {a.positions, ints}, {a.slots, ints}})
               ? CFA_OK
               : CFA_ERR_INVALID_ARG;
}

// The scale (0: the default one) with the exponential's change to base 2.
float scale_log2(float scale) {
    const double s = scale > 0.0f ? scale : 1.0 / std::sqrt(static_cast<double>(kLatQ));
    return static_cast<float>(s * 1.4426950408889634);
}

bool scale_ok(float scale) { return scale >= 0.0f && std::isfinite(scale_log2(scale)); }

cfa_status check_attention(const cfa_latent *p, const AttnArgs &a) {
    if (!a.q || !a.cu || !a.tables || !a.lens || !a.pages || !a.out || a.n_seqs < 1 || a.n_seqs > p->max_seqs ||
        a.n_pages < 1 || cache_rows(p, a.n_pages) < 0 || a.width < 1 || a.width > cfa::kPagedMaxTableWidth ||
        static_cast<long long>(a.width) * p->ps > (1 << 30) || !scale_ok(a.scale))
        return CFA_ERR_INVALID_ARG;
    if (!aligned_to(16, {a.q, a.pages, a.out}) || !aligned_to(4, {a.cu, a.tables, a.lens, a.lse}))
        return CFA_ERR_ALIGNMENT;
    const size_t B4 = 4u * static_cast<size_t>(a.n_seqs);
    return apart({{a.out, heads_bytes(p, a.n_tokens, kLatC)}, {a.lse, a.lse ? heads_bytes(p, a.n_tokens, 2) : 0}},
                 {{a.q, heads_bytes(p, a.n_tokens, kLatRow)}, {a.cu, B4 + 4}, {a.tables, B4 * a.width}, {a.lens, B4},
                  {a.pages, page_bytes(p, a.n_pages)}})
               ? CFA_OK
               : CFA_ERR_INVALID_ARG;
}

cfa_status launch(const void *kernel, dim3 grid, int threads, size_t smem, void *stream, void **args, int cluster = 1) {
    return cfa::launch_kernel(kernel, grid, threads, smem, static_cast<cudaStream_t>(stream), args, cluster);
}

cfa_status launch_append(cfa_latent *p, const AppendArgs &a, void *stream) {
    cfa::LatentAppendParams kp{};
    kp.a = static_cast<const uint16_t *>(a.a);
    kp.g_kv = static_cast<const uint16_t *>(a.g);
    kp.q = static_cast<const uint16_t *>(a.q);
    kp.a_stride = a.as;
    kp.q_stride = a.qs;
    kp.positions = a.positions;
    kp.slots = a.slots;
    kp.pages = static_cast<uint16_t *>(a.pages);
    kp.q_out = static_cast<uint16_t *>(a.q_out);
    kp.status = p->words;
    kp.n_heads = p->nh;
    kp.n_rows = static_cast<int>(cache_rows(p, a.n_pages));
    kp.copy = !in_place(p, a);
    kp.rope = p->rope;
    kp.eps = a.eps;
    kp.magnitude = p->magnitude;
    std::memcpy(kp.turns, p->turns, sizeof kp.turns);
    void *args[1] = {&kp};
    const unsigned parts = 1u + (static_cast<unsigned>(p->nh) + cfa::kLatAppendHeads - 1) / cfa::kLatAppendHeads;
    return launch(cfa::latent_append_kernel_ptr(p->interleaved != 0), dim3(static_cast<unsigned>(a.n_tokens), parts),
                  cfa::kLatAppendThreads, 0, stream, args);
}

// The folding product: x rows of each head, xs elements between tokens.
cfa_status launch_heads(cfa_latent *p, bool fold, int T, const void *x, long long xs, const void *w, void *y, void *stream) {
    cfa::LatentHeadsParams kp{static_cast<const uint16_t *>(x), xs, static_cast<const uint16_t *>(w),
                              static_cast<uint16_t *>(y), T, p->nh, p->words, kTimeoutNs};
    // Few tokens go to many small blocks, which read the weights once for 16 of them; many to tcgen05, which reads
    // them once but takes 1 us more to begin. By 16 tokens times heads, in us, in (few, many): 32 heads, 128 tokens
    // (256) 6.1 and 6.9, 200 (416) 7.6 and 6.5; 128 heads, 48 (384) 7.9 and 8.9, 100 (896) 12.4 and 9.3. Out: 32 heads,
    // 64 (128) 4.6 and 6.4, 100 (224) 7.2 and 6.6; 128 heads, 16 (128) 6.1 and 7.8, 32 (256) 8.9 and 7.9.
    const long long work = (T + cfa::kHeadsTokens - 1ll) / cfa::kHeadsTokens * p->nh;
    if (work <= (fold ? 384 : 160)) {
        void *args[1] = {&kp};
        return launch(cfa::latent_heads_kernel_ptr(fold),
                      dim3(static_cast<unsigned>((T + cfa::kHeadsTokens - 1) / cfa::kHeadsTokens), static_cast<unsigned>(p->nh), 4),
                      128, static_cast<size_t>(cfa::latent_heads_smem(fold)), stream, args);
    }
    const uint64_t H = static_cast<uint64_t>(p->nh), in = H * (fold ? kLatQ : kLatC), out = H * (fold ? kLatRow : kLatV),
                   rows = static_cast<uint64_t>(T);
    CUtensorMap tx, tw, ty;
    if (cfa::encode_bf16_2d_ex(&tx, x, in, rows, static_cast<uint64_t>(xs), 64, 128, true) != CFA_OK ||
        cfa::encode_bf16_2d_ex(&tw, w, H * kLatKv, kLatC, H * kLatKv, 64, 64, true) != CFA_OK ||
        cfa::encode_bf16_2d_ex(&ty, y, out, rows, out, 64, 128, true) != CFA_OK)
        return CFA_ERR_CUDA;
    void *args[4] = {&tx, &tw, &ty, &kp};
    const long long jobs = static_cast<long long>(p->nh) * (fold ? 2 : 1) * ((T + 127) / 128);
    return launch(cfa::latent_heads_mma_kernel_ptr(fold),
                  dim3(static_cast<unsigned>(std::min<long long>(jobs, p->num_sms))), cfa::kHeadsMmaThreads,
                  static_cast<size_t>(cfa::latent_heads_mma_smem(fold)), stream, args);
}

cfa_status launch_fold(cfa_latent *p, int T, const void *q, long long qs, const void *w, void *y, void *stream) {
    return launch_heads(p, true, T, q, qs, w, y, stream);
}

cfa_status launch_unfold(cfa_latent *p, int T, const void *o, const void *w, void *y, void *stream) {
    return launch_heads(p, false, T, o, static_cast<long long>(p->nh) * kLatC, w, y, stream);
}

// Lets the kernels have the shared memory that they ask for.
bool allow_smem() {
    auto allow = [](const void *kernel, int bytes) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
    };
    bool ok = allow(cfa::latent_attention_kernel_ptr(), cfa::latent_attention_smem()) &&
              allow(cfa::latent_expanded_kernel_ptr(), cfa::latent_expanded_smem());
    for (const bool fold : {false, true})
        ok = ok && allow(cfa::latent_heads_kernel_ptr(fold), cfa::latent_heads_smem(fold)) &&
             allow(cfa::latent_heads_mma_kernel_ptr(fold), cfa::latent_heads_mma_smem(fold));
    return ok;
}

cfa_status launch_attention(cfa_latent *p, const AttnArgs &a, void *stream) {
    cfa::LatentAttnParams kp{};
    kp.cu = a.cu;
    kp.lens = a.lens;
    kp.tables = a.tables;
    kp.q = static_cast<const uint16_t *>(a.q);
    kp.pages = static_cast<const uint16_t *>(a.pages);
    kp.out = static_cast<uint16_t *>(a.out);
    kp.lse = a.lse;
    kp.status = p->words;
    kp.T = a.n_tokens;
    kp.B = a.n_seqs;
    kp.H = p->nh;
    kp.page_size = p->ps;
    kp.n_pages = a.n_pages;
    kp.width = a.width;
    kp.scale_log2 = scale_log2(a.scale);
    kp.timeout_ns = kTimeoutNs;
    kp.rec_o = p->rec_o;
    kp.rec_ml = p->rec_ml;
    kp.cuts = p->cuts;
    kp.runs = p->runs;
    kp.by_H = cfa::FastDiv(static_cast<uint32_t>(p->nh));
    kp.by_page = cfa::FastDiv(static_cast<uint32_t>(p->ps));
    kp.box_rows = std::min(p->ps, 64);  // a box lies inside one page and divides 64 keys
    CUtensorMap tq, tr;
    if (cfa::encode_bf16_2d_ex(&tq, a.q, kLatRow, static_cast<uint64_t>(a.n_tokens) * p->nh, kLatRow, 64, 64, true) !=
            CFA_OK ||
        cfa::encode_bf16_2d_ex(&tr, a.pages, kLatRow, static_cast<uint64_t>(cache_rows(p, a.n_pages)), kLatRow, 64,
                               static_cast<uint32_t>(kp.box_rows), true) != CFA_OK)
        return CFA_ERR_CUDA;
    void *args[3] = {&tq, &tr, &kp};
    const cfa_status st = launch(cfa::latent_attention_kernel_ptr(), dim3(2u * static_cast<unsigned>(p->runs)),
                                 cfa::kLatAttnThreads, static_cast<size_t>(cfa::latent_attention_smem()), stream, args);
    if (st != CFA_OK) return st;
    void *margs[1] = {&kp};
    return launch(cfa::latent_merge_kernel_ptr(), dim3(2u * static_cast<unsigned>(p->num_sms)),
                  cfa::kLatMergeThreads, 0, stream, margs);
}

}  // namespace

extern "C" {

cfa_latent *cfa_latent_create(int max_seqs, int max_tokens, int n_heads, int page_size) {
    if (max_seqs < 1 || max_tokens < 1 || n_heads < 1 || page_size < 1) {
        fail(CFA_ERR_INVALID_ARG);
        return nullptr;
    }
    if (max_seqs > cfa::kPagedMaxSeqs || max_tokens > cfa::kPagedMaxTokens || n_heads > 1024 || page_size > (1 << 22) ||
        (page_size != 16 && page_size != 32 && page_size % 64)) {
        fail(CFA_ERR_UNSUPPORTED);
        return nullptr;
    }
    int device = -1, major = 0, minor = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
        cudaGetLastError();
        fail(CFA_ERR_CUDA);
        return nullptr;
    }
    if (major != 10 || minor != 3) {  // built for sm_103a only
        fail(CFA_ERR_UNSUPPORTED);
        return nullptr;
    }
    cfa_latent *p = new (std::nothrow) cfa_latent();
    if (!p) {
        fail(CFA_ERR_CUDA);
        return nullptr;
    }
    p->max_seqs = max_seqs;
    p->max_tokens = max_tokens;
    p->nh = n_heads;
    p->ps = page_size;
    p->device = device;
    p->num_sms = sms;
    p->runs = std::min(sms / 2, cfa::kLatMaxRuns);
    const size_t rec_rows = 2u * static_cast<size_t>(p->runs) * cfa::kLatTile;
    if (!allow_smem() ||
        cudaMalloc(&p->words, cfa::kLatWords * sizeof(unsigned)) != cudaSuccess || !clear_words(p->words, cfa::kLatWords) ||
        cudaMalloc(&p->rec_o, sizeof(float) * rec_rows * kLatC) != cudaSuccess ||
        // (twice the rows: the expanded form's records are 512 rows of 128 dims, one a cluster)
        cudaMalloc(&p->rec_ml, 2 * sizeof(float2) * rec_rows) != cudaSuccess ||
        // (twice the runs: two tiles of a split task)
        cudaMalloc(&p->cuts, 2 * sizeof(int4) * static_cast<size_t>(p->runs)) != cudaSuccess) {
        cudaGetLastError();
        latent_free(p);
        delete p;
        fail(CFA_ERR_CUDA);
        return nullptr;
    }
    return p;
}

void cfa_latent_destroy(cfa_latent *p) {
    if (!p) return;
    OnDevice on(p->device);
    cudaDeviceSynchronize();
    latent_free(p);
    delete p;
}

cfa_status cfa_latent_set_rope(cfa_latent *p, double theta, int interleaved, int scaling, double factor,
                               double low_turns, double high_turns, int original_ctx, double magnitude) {
    if (!p) return fail(CFA_ERR_INVALID_ARG);
    if (theta == 0.0) {
        p->rope = 0;
        return CFA_OK;
    }
    unsigned long long turns[kLatR / 2];
    const cfa_status st = cfa::rope_turns(theta, kLatR, scaling, factor, low_turns, high_turns, original_ctx,
                                          magnitude, turns);
    if (st != CFA_OK) return fail(st);
    std::memcpy(p->turns, turns, sizeof turns);
    p->rope = 1;
    p->interleaved = interleaved ? 1 : 0;
    p->scaling = scaling;
    p->magnitude = static_cast<float>(magnitude);
    return CFA_OK;
}

cfa_status cfa_latent_append(cfa_latent *p, int n_tokens, const void *a, long long a_stride, const void *g_kv,
                             float eps, const void *q, long long q_stride, const int *positions, const int *slots,
                             int n_pages, void *pages, void *q_out, void *stream) {
    if (!p || !tokens_ok(p, n_tokens)) return fail(CFA_ERR_INVALID_ARG);
    if (n_tokens == 0) return CFA_OK;
    const AppendArgs x{n_tokens, a, a_stride, g_kv, eps, q, q_stride, positions, slots, n_pages, pages, q_out};
    cfa_status st = check_append(p, x);
    if (st != CFA_OK) return fail(st);
    OnDevice on(p->device);
    if (!on.ok()) return fail(CFA_ERR_CUDA);
    st = launch_append(p, x, stream);
    return st == CFA_OK ? CFA_OK : fail(st);
}

cfa_status cfa_latent_fold(cfa_latent *p, int n_tokens, const void *q, long long q_stride, const void *W_kvb,
                           void *q_lat, void *stream) {
    if (!p || !tokens_ok(p, n_tokens)) return fail(CFA_ERR_INVALID_ARG);
    if (n_tokens == 0) return CFA_OK;
    const long long wide = static_cast<long long>(p->nh) * kLatQ;
    if (!q || !W_kvb || !q_lat || !stride_ok(wide, q_stride)) return fail(CFA_ERR_INVALID_ARG);
    if (!aligned_to(16, {q, W_kvb, q_lat})) return fail(CFA_ERR_ALIGNMENT);
    if (!apart({{q_lat, heads_bytes(p, n_tokens, kLatRow)}},
               {{q, span(n_tokens, wide, q_stride)}, {W_kvb, weight_bytes(p)}}))
        return fail(CFA_ERR_INVALID_ARG);
    OnDevice on(p->device);
    if (!on.ok()) return fail(CFA_ERR_CUDA);
    const cfa_status st = launch_fold(p, n_tokens, q, q_stride, W_kvb, q_lat, stream);
    return st == CFA_OK ? CFA_OK : fail(st);
}

cfa_status cfa_latent_unfold(cfa_latent *p, int n_tokens, const void *o_lat, const void *W_kvb, void *out,
                             void *stream) {
    if (!p || !tokens_ok(p, n_tokens)) return fail(CFA_ERR_INVALID_ARG);
    if (n_tokens == 0) return CFA_OK;
    if (!o_lat || !W_kvb || !out) return fail(CFA_ERR_INVALID_ARG);
    if (!aligned_to(16, {o_lat, W_kvb, out})) return fail(CFA_ERR_ALIGNMENT);
    if (!apart({{out, heads_bytes(p, n_tokens, kLatV)}},
               {{o_lat, heads_bytes(p, n_tokens, kLatC)}, {W_kvb, weight_bytes(p)}}))
        return fail(CFA_ERR_INVALID_ARG);
    OnDevice on(p->device);
    if (!on.ok()) return fail(CFA_ERR_CUDA);
    const cfa_status st = launch_unfold(p, n_tokens, o_lat, W_kvb, out, stream);
    return st == CFA_OK ? CFA_OK : fail(st);
}

cfa_status cfa_latent_attention(cfa_latent *p, int n_tokens, int n_seqs, const void *q_lat, const int *cu,
                                const int *tables, int table_width, const int *lens, int n_pages, const void *pages,
                                float scale, void *o_lat, float *lse, void *stream) {
    if (!p || !tokens_ok(p, n_tokens)) return fail(CFA_ERR_INVALID_ARG);
    if (n_tokens == 0) return CFA_OK;
    const AttnArgs x{n_tokens, n_seqs, q_lat, cu, tables, table_width, lens, n_pages, pages, scale, o_lat, lse};
    cfa_status st = check_attention(p, x);
    if (st != CFA_OK) return fail(st);
    OnDevice on(p->device);
    if (!on.ok()) return fail(CFA_ERR_CUDA);
    st = launch_attention(p, x, stream);
    return st == CFA_OK ? CFA_OK : fail(st);
}

cfa_status cfa_latent_expanded(cfa_latent *p, int n_tokens, int n_keys, int n_seqs, const void *q,
                               long long q_stride, const void *kv, long long kv_stride, const void *k_rope,
                               long long k_rope_stride, const int *cu, const int *cu_k, float scale, void *out,
                               float *lse, void *stream) {
    if (!p || !tokens_ok(p, n_tokens)) return fail(CFA_ERR_INVALID_ARG);
    if (n_tokens == 0) return CFA_OK;
    const long long wide = static_cast<long long>(p->nh) * kLatQ, kwide = static_cast<long long>(p->nh) * kLatKv;
    if (!q || !cu || !cu_k || !out || n_seqs < 1 || n_seqs > p->max_seqs || n_keys < 0 || n_keys > (1 << 30) ||
        !stride_ok(wide, q_stride) || !scale_ok(scale) ||
        (n_keys > 0 && (!kv || !k_rope || !stride_ok(kwide, kv_stride) || !stride_ok(kLatR, k_rope_stride))))
        return fail(CFA_ERR_INVALID_ARG);
    if (!aligned_to(16, {q, kv, k_rope, out}) || !aligned_to(4, {cu, cu_k, lse})) return fail(CFA_ERR_ALIGNMENT);
    const size_t B4 = 4u * static_cast<size_t>(n_seqs) + 4;
    if (!apart({{out, heads_bytes(p, n_tokens, kLatV)}, {lse, lse ? heads_bytes(p, n_tokens, 2) : 0}},
               {{q, span(n_tokens, wide, q_stride)}, {cu, B4}, {cu_k, B4}, {kv, span(n_keys, kwide, kv_stride)},
                {k_rope, span(n_keys, kLatR, k_rope_stride)}}))
        return fail(CFA_ERR_INVALID_ARG);
    OnDevice on(p->device);
    if (!on.ok()) return fail(CFA_ERR_CUDA);
    cfa::LatentExpandedParams kp{};
    kp.kv = static_cast<const uint16_t *>(kv);
    kp.kv_stride = kv_stride;
    kp.cu = cu;
    kp.cu_k = cu_k;
    kp.out = static_cast<uint16_t *>(out);
    kp.lse = lse;
    kp.status = p->words;
    kp.odd = p->words + 1;
    kp.odd_tiles = reinterpret_cast<unsigned char *>(p->words + 4);
    kp.rec_o = p->rec_o;
    kp.rec_ml = p->rec_ml;
    kp.T = n_tokens;
    kp.S = n_keys;
    kp.B = n_seqs;
    kp.H = p->nh;
    kp.rest = reinterpret_cast<int *>(p->words + 3);
    kp.splits = p->cuts;
    kp.by_H = cfa::FastDiv(static_cast<uint32_t>(p->nh));
    kp.scale_log2 = scale_log2(scale);
    kp.timeout_ns = kTimeoutNs;
    // without keys the kernel loads none: any map will do
    const uint64_t rows = static_cast<uint64_t>(std::max(n_keys, 1));
    CUtensorMap tq, tk, tr;
    if (cfa::encode_bf16_2d_ex(&tq, q, static_cast<uint64_t>(wide), static_cast<uint64_t>(n_tokens),
                               static_cast<uint64_t>(q_stride), 64, 128, true) != CFA_OK ||
        cfa::encode_bf16_2d_ex(&tk, n_keys ? kv : q, static_cast<uint64_t>(n_keys ? kwide : 64), rows,
                               static_cast<uint64_t>(n_keys ? kv_stride : 64), 64, 64, true) != CFA_OK ||
        cfa::encode_bf16_2d_ex(&tr, n_keys ? k_rope : q, kLatR, rows, static_cast<uint64_t>(n_keys ? k_rope_stride : 64),
                               64, 64, true) != CFA_OK)
        return fail(CFA_ERR_CUDA);
    void *args[4] = {&tq, &tk, &tr, &kp};
    cfa_status st = launch(cfa::latent_expanded_kernel_ptr(), dim3(2u * static_cast<unsigned>(p->runs)), cfa::kExpThreads,
                           static_cast<size_t>(cfa::latent_expanded_smem()), stream, args);
    void *margs[1] = {&kp};
    if (st == CFA_OK)
        st = launch(cfa::latent_expanded_merge_kernel_ptr(), dim3(2u * static_cast<unsigned>(p->num_sms)),
                    cfa::kLatMergeThreads, 0, stream, margs);
    return st == CFA_OK ? CFA_OK : fail(st);
}

cfa_status cfa_latent_layer(cfa_latent *p, int n_tokens, int n_seqs, const void *a, long long a_stride,
                            const void *g_kv, float eps, const void *q, long long q_stride, const int *positions,
                            const int *slots, const int *cu, const int *tables, int table_width, const int *lens,
                            int n_pages, void *pages, const void *W_kvb, float scale, void *q_out, void *q_lat,
                            void *o_lat, float *lse, void *out, void *stream) {
    if (!p || !tokens_ok(p, n_tokens)) return fail(CFA_ERR_INVALID_ARG);
    if (n_tokens == 0) return CFA_OK;
    const AppendArgs x{n_tokens, a, a_stride, g_kv, eps, q, q_stride, positions, slots, n_pages, pages, q_out};
    const AttnArgs y{n_tokens, n_seqs, q_lat, cu, tables, table_width, lens, n_pages, pages, scale, o_lat, lse};
    cfa_status st = check_append(p, x);
    if (st == CFA_OK) st = check_attention(p, y);
    if (st != CFA_OK) return fail(st);
    if (!W_kvb || !out) return fail(CFA_ERR_INVALID_ARG);
    if (!aligned_to(16, {W_kvb, out})) return fail(CFA_ERR_ALIGNMENT);
    // and what neither check sees: every array that the call writes lies apart from all others
    const size_t ints = 4u * static_cast<size_t>(n_tokens), B4 = 4u * static_cast<size_t>(n_seqs);
    const long long wide = static_cast<long long>(p->nh) * kLatQ;
    if (!apart({{pages, page_bytes(p, n_pages)}, {q_out, heads_bytes(p, n_tokens, kLatQ)},
                {q_lat, heads_bytes(p, n_tokens, kLatRow)}, {o_lat, heads_bytes(p, n_tokens, kLatC)},
                {lse, lse ? heads_bytes(p, n_tokens, 2) : 0}, {out, heads_bytes(p, n_tokens, kLatV)}},
               {{a, span(n_tokens, kLatRow, a_stride)}, {g_kv, 2 * kLatC},
                {q, in_place(p, x) ? 0 : span(n_tokens, wide, q_stride)}, {positions, ints}, {slots, ints},
                {cu, B4 + 4}, {tables, B4 * table_width}, {lens, B4}, {W_kvb, weight_bytes(p)}}))
        return fail(CFA_ERR_INVALID_ARG);
    OnDevice on(p->device);
    if (!on.ok()) return fail(CFA_ERR_CUDA);
    st = launch_append(p, x, stream);
    if (st == CFA_OK) st = launch_fold(p, n_tokens, q_out, wide, W_kvb, q_lat, stream);
    if (st == CFA_OK) st = launch_attention(p, y, stream);
    if (st == CFA_OK) st = launch_unfold(p, n_tokens, o_lat, W_kvb, out, stream);
    return st == CFA_OK ? CFA_OK : fail(st);
}

cfa_status cfa_latent_status(cfa_latent *p) {
    if (!p) return fail(CFA_ERR_INVALID_ARG);
    OnDevice on(p->device);
    unsigned v = 0;
    if (!on.ok() || cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(&v, p->words, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess || !clear_words(p->words, 1)) {
        cudaGetLastError();
        return fail(CFA_ERR_CUDA);
    }
    if (v & cfa::kStatusTimeoutBit) return fail(CFA_ERR_TIMEOUT);
    if (v & (cfa::kStatusBadLengthBit | cfa::kStatusBadPageBit)) return fail(CFA_ERR_INVALID_ARG);
    return CFA_OK;
}

cfa_status cfa_latent_describe(const cfa_latent *p, char *buf, int len) {
    if (!p || !buf || len < 1) return fail(CFA_ERR_INVALID_ARG);
    std::snprintf(buf, static_cast<size_t>(len),
                  "{\"max_seqs\": %d, \"max_tokens\": %d, \"n_heads\": %d, \"page_size\": %d, \"rope\": %d, "
                  "\"interleaved\": %d, \"scaling\": %d, \"num_sms\": %d, \"runs\": %d, \"smem_bytes\": %d, "
                  "\"workspace_bytes\": %lld}",
                  p->max_seqs, p->max_tokens, p->nh, p->ps, p->rope, p->interleaved, p->scaling, p->num_sms, p->runs,
                  cfa::latent_attention_smem(), 2ll * p->runs * cfa::kLatTile * (4 * kLatC + 16) + 32ll * p->runs + cfa::kExpMarks);
    return CFA_OK;
}

}  // extern "C"
