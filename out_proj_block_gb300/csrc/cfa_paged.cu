// cfa_paged.cu -- host side of the paged-cache entry points (include/cfa.h):
// argument checks, the rotation's frequencies, the workspace and the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <new>

#include "cfa.h"
#include "cfa_host.h"
#include "cfa_internal.h"
#include "cfa_paged.h"
#include "cfa_paged_split.h"

namespace cfa {
const void *paged_tables_kernel_ptr();
const void *paged_append_kernel_ptr(bool interleaved);
const void *paged_attention_kernel_ptr(int d);
const void *paged_merge_kernel_ptr(int d);
int paged_attention_smem(int d, int seqs);
}  // namespace cfa

struct cfa_paged {
    int max_seqs = 0, max_tokens = 0, nh = 0, nkv = 0, D = 0, ps = 0;
    int device = -1, num_sms = 0;
    // rotation
    int rd = 0, interleaved = 0, scaling = CFA_ROPE_PLAIN;
    float magnitude = 1.0f;
    unsigned long long turns[64] = {};
    // workspace
    unsigned *words = nullptr;  // [0] status, [1] arrivals of the tables' blocks, [2..3] the merge's (odd)
    int *plan_ws = nullptr;     // the attention's scan, for its merge
    float *rec_o = nullptr;     // records of the attention's pieces
    float2 *rec_ml = nullptr;
    long long rec_rows = 0;
    size_t plan_ints = 0;
};

namespace {

constexpr uint32_t kTimeoutNs = 2000000000u;  // 2 s per device-side wait

cfa_status fail(cfa_status s) { return cfa::set_last_error(s); }

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

// The plan's device is the current one for the length of a call.
class OnDevice {
  public:
    explicit OnDevice(int device) {
        if (cudaGetDevice(&was_) != cudaSuccess) was_ = -1;
        ok_ = was_ == device || cudaSetDevice(device) == cudaSuccess;
        if (was_ == device) was_ = -1;
        if (!ok_) cudaGetLastError();
    }
    ~OnDevice() {
        if (was_ >= 0) cudaSetDevice(was_);
    }
    bool ok() const { return ok_; }

  private:
    int was_ = -1;
    bool ok_ = false;
};

cfa_status launch(const void *kernel, int grid, int threads, size_t smem, cudaStream_t stream,
                  void **args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
        cudaGetLastError();
        return CFA_ERR_CUDA;
    }
    return CFA_OK;
}

void paged_free(cfa_paged *p) {
    if (p->words) cudaFree(p->words);
    if (p->plan_ws) cudaFree(p->plan_ws);
    if (p->rec_o) cudaFree(p->rec_o);
    if (p->rec_ml) cudaFree(p->rec_ml);
    p->words = nullptr;
    p->plan_ws = nullptr;
    p->rec_o = nullptr;
    p->rec_ml = nullptr;
}

// Clears words of a plan. A memset may run after the call that asks for it has returned, and
// streams that do not wait for the legacy one would launch on what the words held before.
bool clear_words(unsigned *words, int n) {
    return cudaMemset(words, 0, sizeof(unsigned) * n) == cudaSuccess && cudaStreamSynchronize(nullptr) == cudaSuccess;
}

// Rows of a cache of n_pages pages, or -1 where they pass the kernels' 32-bit
// row index.
long long cache_rows(const cfa_paged *p, int n_pages) {
    const long long rows = static_cast<long long>(n_pages) * p->nkv;
    return rows > ((1ll << 31) - 1) / p->ps ? -1 : rows * p->ps;
}

struct AppendArgs {
    int n_tokens;
    const void *q, *k, *v;
    long long qs, ks, vs;
    const int *positions, *slots;
    int n_pages;
    void *kp, *vp, *q_out;
};

struct AttnArgs {
    int n_tokens, n_seqs;
    const void *q;
    long long qs;
    const int *cu, *prefix_table;
    int prefix_len;
    const int *tables;
    int width;
    const int *lens;
    int n_pages;
    const void *kp, *vp;
    float scale;
    void *out;
    float *lse;
};

// Bytes that n rows of `heads` heads with this stride span.
size_t span(const cfa_paged *p, int n, int heads, long long stride) {
    return n ? 2u * (static_cast<size_t>(n - 1) * static_cast<size_t>(stride) +
                     static_cast<size_t>(heads) * p->D)
             : 0;
}

bool stride_ok(const cfa_paged *p, int heads, long long stride) {
    return stride >= static_cast<long long>(heads) * p->D && stride % 8 == 0 && stride < (1ll << 40);
}

cfa_status check_append(const cfa_paged *p, const AppendArgs &a) {
    if (a.n_tokens == 0) return CFA_OK;  // nothing to do
    if (!a.q || !a.k || !a.v || !a.positions || !a.slots || !a.kp || !a.vp || !a.q_out ||
        a.n_tokens < 0 || a.n_tokens > p->max_tokens || a.n_pages < 1 || cache_rows(p, a.n_pages) < 0 ||
        !stride_ok(p, p->nh, a.qs) || !stride_ok(p, p->nkv, a.ks) || !stride_ok(p, p->nkv, a.vs))
        return CFA_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.kp, 16) ||
        !aligned(a.vp, 16) || !aligned(a.q_out, 16) || !aligned(a.positions, 4) || !aligned(a.slots, 4))
        return CFA_ERR_ALIGNMENT;
    const long long dense = static_cast<long long>(p->nh) * p->D;
    const size_t nq = span(p, a.n_tokens, p->nh, a.qs), nk = span(p, a.n_tokens, p->nkv, a.ks),
                 nv = span(p, a.n_tokens, p->nkv, a.vs), no = span(p, a.n_tokens, p->nh, dense),
                 pages = 2u * static_cast<size_t>(cache_rows(p, a.n_pages)) * p->D,
                 ints = 4u * static_cast<size_t>(a.n_tokens);
    if ((overlaps(a.q_out, no, a.q, nq) && !(a.q_out == a.q && a.qs == dense)) ||
        overlaps(a.q_out, no, a.k, nk) || overlaps(a.q_out, no, a.v, nv) ||
        overlaps(a.kp, pages, a.vp, pages))
        return CFA_ERR_INVALID_ARG;
    const void *cache[2] = {a.kp, a.vp};
    for (const void *c : cache)
        if (overlaps(c, pages, a.q, nq) || overlaps(c, pages, a.k, nk) || overlaps(c, pages, a.v, nv) ||
            overlaps(c, pages, a.q_out, no) || overlaps(c, pages, a.positions, ints) ||
            overlaps(c, pages, a.slots, ints))
            return CFA_ERR_INVALID_ARG;
    if (overlaps(a.q_out, no, a.positions, ints) || overlaps(a.q_out, no, a.slots, ints))
        return CFA_ERR_INVALID_ARG;
    return CFA_OK;
}

// The scale (0: the default one) with the exponential's change to base 2.
float scale_log2(const cfa_paged *p, float scale) {
    const double s = scale > 0.0f ? scale : 1.0 / std::sqrt(static_cast<double>(p->D));
    return static_cast<float>(s * 1.4426950408889634);
}

struct Span {
    const void *at;
    size_t n;
};

// Whether n bytes at `out` lie over the arrays that say what the batch is.
bool over_batch(const cfa_paged *p, const AttnArgs &a, const void *out, size_t n) {
    const Span in[] = {
        {a.cu, 4u * (static_cast<size_t>(a.n_seqs) + 1)},
        {a.lens, 4u * static_cast<size_t>(a.n_seqs)},
        {a.tables, 4u * static_cast<size_t>(a.n_seqs) * a.width},
        {a.prefix_table, a.prefix_len ? 4u * ((static_cast<size_t>(a.prefix_len) + p->ps - 1) / p->ps) : 0}};
    for (const Span &b : in)
        if (overlaps(out, n, b.at, b.n)) return true;
    return false;
}

cfa_status check_attention(const cfa_paged *p, const AttnArgs &a) {
    if (a.n_tokens == 0) return CFA_OK;  // nothing to do
    if (!a.q || !a.cu || !a.tables || !a.lens || !a.kp || !a.vp || !a.out || a.n_tokens < 0 ||
        a.n_tokens > p->max_tokens || a.n_seqs < 1 || a.n_seqs > p->max_seqs || a.n_pages < 1 ||
        cache_rows(p, a.n_pages) < 0 || !stride_ok(p, p->nh, a.qs) || a.prefix_len < 0 ||
        a.prefix_len > (1 << 30) || (a.prefix_len > 0 && !a.prefix_table) || a.width < 1 ||
        a.width > cfa::kPagedMaxTableWidth ||
        static_cast<long long>(a.width) * p->ps > (1 << 30) || !(a.scale >= 0.0f) ||
        !std::isfinite(scale_log2(p, a.scale)))
        return CFA_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.kp, 16) || !aligned(a.vp, 16) || !aligned(a.out, 16) ||
        !aligned(a.cu, 4) || !aligned(a.prefix_table, 4) || !aligned(a.tables, 4) ||
        !aligned(a.lens, 4) || !aligned(a.lse, 4))
        return CFA_ERR_ALIGNMENT;
    const size_t no = span(p, a.n_tokens, p->nh, static_cast<long long>(p->nh) * p->D);
    const size_t nl = a.lse ? 4u * static_cast<size_t>(a.n_tokens) * p->nh : 0;
    const size_t pages = 2u * static_cast<size_t>(cache_rows(p, a.n_pages)) * p->D;
    const Span q_and_cache[] = {{a.q, span(p, a.n_tokens, p->nh, a.qs)}, {a.kp, pages}, {a.vp, pages}};
    for (const Span &b : q_and_cache)
        if (overlaps(a.out, no, b.at, b.n) || overlaps(a.lse, nl, b.at, b.n)) return CFA_ERR_INVALID_ARG;
    if (over_batch(p, a, a.out, no) || over_batch(p, a, a.lse, nl)) return CFA_ERR_INVALID_ARG;
    return overlaps(a.out, no, a.lse, nl) ? CFA_ERR_INVALID_ARG : CFA_OK;
}

// Both calls' checks, and what neither sees: the append writes before the attention reads its
// offsets and tables, and the next layer's call reads the positions and slots again.
cfa_status check_layer(const cfa_paged *p, const AppendArgs &a, const AttnArgs &b) {
    cfa_status st = check_append(p, a);
    if (st == CFA_OK) st = check_attention(p, b);
    if (st != CFA_OK || a.n_tokens == 0) return st;
    const size_t no = span(p, a.n_tokens, p->nh, static_cast<long long>(p->nh) * p->D);
    const size_t pages = 2u * static_cast<size_t>(cache_rows(p, a.n_pages)) * p->D;
    if (over_batch(p, b, a.q_out, no) || over_batch(p, b, a.kp, pages) || over_batch(p, b, a.vp, pages))
        return CFA_ERR_INVALID_ARG;
    const size_t nl = b.lse ? 4u * static_cast<size_t>(a.n_tokens) * p->nh : 0;
    const size_t ints = 4u * static_cast<size_t>(a.n_tokens);
    for (const int *t : {a.positions, a.slots})
        if (overlaps(b.out, no, t, ints) || overlaps(b.lse, nl, t, ints)) return CFA_ERR_INVALID_ARG;
    return CFA_OK;
}

// Threads of an append block, which takes a token's rows of q, k and v: 64 up to 16 KB of
// them, 128 above (60 MB of rows, read and written: 6 KB a token 21.3 and 23.9 us, 12 KB 20.7
// and 21.8, 16 KB 20.4 and 20.6, 18 KB 22.1 and 20.6, 24 KB 23.6 and 20.9).
int append_threads(const cfa_paged *p) { return (p->nh + 2 * p->nkv) * p->D * 2 <= 16384 ? 64 : cfa::kAppendThreads; }

cfa_status launch_append(cfa_paged *p, const AppendArgs &a, cudaStream_t stream) {
    if (a.n_tokens == 0) return CFA_OK;
    cfa::AppendParams kp{};
    kp.q = static_cast<const uint16_t *>(a.q);
    kp.k = static_cast<const uint16_t *>(a.k);
    kp.v = static_cast<const uint16_t *>(a.v);
    kp.q_stride = a.qs;
    kp.k_stride = a.ks;
    kp.v_stride = a.vs;
    kp.positions = a.positions;
    kp.slots = a.slots;
    kp.k_pages = static_cast<uint16_t *>(a.kp);
    kp.v_pages = static_cast<uint16_t *>(a.vp);
    kp.q_out = static_cast<uint16_t *>(a.q_out);
    kp.status = p->words;
    kp.n_heads = p->nh;
    kp.n_kv = p->nkv;
    kp.d = p->D;
    kp.page_size = p->ps;
    kp.n_rows = a.n_pages * p->ps;
    kp.rd = p->rd;
    kp.interleaved = p->interleaved;
    kp.by_units = cfa::FastDiv(static_cast<uint32_t>((p->interleaved ? p->rd / 8 : p->rd / 16) + (p->D - p->rd) / 8));
    kp.heads_a_pass = append_threads(p) / static_cast<int>(kp.by_units.d);
    kp.by_page = cfa::FastDiv(static_cast<uint32_t>(p->ps));
    kp.magnitude = p->magnitude;
    std::memcpy(kp.turns, p->turns, sizeof kp.turns);
    void *args[1] = {&kp};
    return launch(cfa::paged_append_kernel_ptr(p->interleaved != 0), a.n_tokens, append_threads(p), 0, stream, args);
}

cfa_status launch_attention(cfa_paged *p, const AttnArgs &a, cudaStream_t stream) {
    if (a.n_tokens == 0) return CFA_OK;
    cfa::PagedAttnParams kp{};
    kp.q = static_cast<const uint16_t *>(a.q);
    kp.q_stride = a.qs;
    kp.v_pages = static_cast<const uint16_t *>(a.vp);
    kp.v_pages = static_cast<const uint16_t *>(a.vp);
    kp.cu = a.cu;
    kp.lens = a.lens;
    kp.tables = a.tables;
    kp.prefix_table = a.prefix_table;
    kp.out = static_cast<uint16_t *>(a.out);
    kp.lse = a.lse;
    kp.status = p->words;
    kp.odd = p->words + 2;
    kp.T = a.n_tokens;
    kp.B = a.n_seqs;
    kp.n_heads = p->nh;
    kp.n_kv = p->nkv;
    kp.page_size = p->ps;
    kp.n_pages = a.n_pages;
    kp.width = a.width;
    kp.prefix_len = a.prefix_len;
    kp.scale_log2 = scale_log2(p, a.scale);
    kp.plan_ws = p->plan_ws;
    kp.rec_o = p->rec_o;
    kp.rec_ml = p->rec_ml;
    kp.timeout_ns = kTimeoutNs;
    // 512 D bytes at 6.8 TB/s over 152 SMs of 1.9 GHz, by 400 clocks: 2780 at head_dim 128. At 64
    // 1390, beside some 1350 of work on a block of few rows that counts as 5 (paged_cost): 5, so
    // that there the bytes never bound the whole. 6 there took 52.1 us instead of 40.0 for 16
    // requests of some 550 keys without a prefix (64 heads) and 68.8 instead of 56.6 for 4 of
    // some 4000, and was nowhere more than 0.7% faster (8 of some 1100 behind 2048).
    kp.block_clocks = p->D == 128 ? 7 : 5;
    kp.shape = cfa::PagedShape(p->nh / p->nkv, p->nkv, a.prefix_len, p->num_sms);
    kp.by_page = cfa::FastDiv(static_cast<uint32_t>(p->ps));
    // a box of rows lies inside one page and divides a block of 128 keys
    kp.box_rows = p->ps % 128 == 0 ? 128 : p->ps % 64 == 0 ? 64 : p->ps;
    CUtensorMap tk, tv;
    const uint64_t rows = static_cast<uint64_t>(cache_rows(p, a.n_pages)), d = static_cast<uint64_t>(p->D);
    if (cfa::encode_bf16_2d_ex(&tk, a.kp, d, rows, d, 64, static_cast<uint32_t>(kp.box_rows), true) != CFA_OK ||
        cfa::encode_bf16_2d_ex(&tv, a.vp, d, rows, d, 64, static_cast<uint32_t>(kp.box_rows), true) != CFA_OK)
        return CFA_ERR_CUDA;
    void *args[3] = {&tk, &tv, &kp};
    const int grid = p->num_sms;
    const cfa_status st = launch(cfa::paged_attention_kernel_ptr(p->D), grid, cfa::kPagedThreads,
                           static_cast<size_t>(cfa::paged_attention_smem(p->D, a.n_seqs)), stream, args);
    if (st != CFA_OK) return st;
    void *margs[1] = {&kp};
    return launch(cfa::paged_merge_kernel_ptr(p->D), 3 * grid, cfa::kPagedMergeThreads, 0, stream, margs);
}

}  // namespace

extern "C" {

cfa_paged *cfa_paged_create(int max_seqs, int max_tokens, int n_heads, int n_kv_heads,
                            int head_dim, int page_size) {
    if (max_seqs < 1 || max_tokens < 1 || n_heads < 1 || n_kv_heads < 1 || head_dim < 1 ||
        page_size < 1 || n_heads % n_kv_heads) {
        fail(CFA_ERR_INVALID_ARG);
        return nullptr;
    }
    if (max_seqs > cfa::kPagedMaxSeqs || max_tokens > cfa::kPagedMaxTokens || n_heads > 1024 ||
        (head_dim != 64 && head_dim != 128) || page_size > (1 << 22) ||
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
    cfa_paged *p = new (std::nothrow) cfa_paged();
    if (!p) {
        fail(CFA_ERR_CUDA);
        return nullptr;
    }
    p->max_seqs = max_seqs;
    p->max_tokens = max_tokens;
    p->nh = n_heads;
    p->nkv = n_kv_heads;
    p->D = head_dim;
    p->ps = page_size;
    p->device = device;
    p->num_sms = std::min(sms, cfa::kPagedMaxGrid);
    const int G = n_heads / n_kv_heads;
    const long long shared = std::min(static_cast<long long>(max_tokens) * G,
                                      static_cast<long long>(max_seqs) * cfa::kPagedAloneRows);
    p->rec_rows = cfa::paged_record_rows(cfa::PagedShape(G, n_kv_heads, 0, p->num_sms), shared);
    p->plan_ints = cfa::kPagedPlanInts + 8 * (static_cast<size_t>(p->num_sms) + static_cast<size_t>(shared));
    if (cudaFuncSetAttribute(cfa::paged_tables_kernel_ptr(), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(int)) * (3 * cfa::kPagedMaxSeqs + 2)) != cudaSuccess ||
        cudaFuncSetAttribute(cfa::paged_attention_kernel_ptr(head_dim), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             cfa::paged_attention_smem(head_dim, cfa::kPagedMaxSeqs)) != cudaSuccess ||
        cudaMalloc(&p->words, 4 * sizeof(unsigned)) != cudaSuccess ||
        !clear_words(p->words, 4) ||
        cudaMalloc(&p->plan_ws, sizeof(int) * p->plan_ints) != cudaSuccess ||
        cudaMalloc(&p->rec_o, sizeof(float) * static_cast<size_t>(p->rec_rows) * head_dim) != cudaSuccess ||
        cudaMalloc(&p->rec_ml, sizeof(float2) * static_cast<size_t>(p->rec_rows)) != cudaSuccess) {
        cudaGetLastError();
        paged_free(p);
        delete p;
        fail(CFA_ERR_CUDA);
        return nullptr;
    }
    return p;
}

void cfa_paged_destroy(cfa_paged *p) {
    if (!p) return;
    OnDevice on(p->device);
    cudaDeviceSynchronize();
    paged_free(p);
    delete p;
}

cfa_status cfa_paged_set_rope(cfa_paged *p, double theta, int rotary_dim, int interleaved,
                              int scaling, double factor, double low_turns, double high_turns,
                              int original_ctx, double magnitude) {
    if (!p || rotary_dim < 0) return fail(CFA_ERR_INVALID_ARG);
    if (rotary_dim > p->D || rotary_dim % 16) return fail(CFA_ERR_UNSUPPORTED);
    if (rotary_dim == 0) {
        p->rd = 0;
        return CFA_OK;
    }
    if (!(theta >= 1.0) || !std::isfinite(theta) || !(factor >= 1.0) || !std::isfinite(factor) ||
        !(magnitude > 0.0) || !std::isfinite(magnitude) || magnitude > 1e6 ||
        scaling < CFA_ROPE_PLAIN || scaling > CFA_ROPE_BY_PARTS)
        return fail(CFA_ERR_INVALID_ARG);
    if (scaling == CFA_ROPE_BY_PARTS &&
        (!(low_turns >= 0.0) || !(high_turns > low_turns) || !std::isfinite(high_turns) || original_ctx < 1))
        return fail(CFA_ERR_INVALID_ARG);
    const double two_pi = 6.283185307179586476925287;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rotary_dim);
        if (scaling == CFA_ROPE_LINEAR) f /= factor;
        if (scaling == CFA_ROPE_BY_PARTS) {
            const double r = original_ctx * f / two_pi;
            const double g = std::min(1.0, std::max(0.0, (r - low_turns) / (high_turns - low_turns)));
            f = g * f + (1.0 - g) * f / factor;
        }
        // f <= 1, so below 1/6 of a turn: the product stays far below 2^64
        p->turns[i] = static_cast<unsigned long long>(std::ldexp(f / two_pi, 64));
    }
    p->rd = rotary_dim;
    p->interleaved = interleaved ? 1 : 0;
    p->scaling = scaling;
    p->magnitude = static_cast<float>(magnitude);
    return CFA_OK;
}

cfa_status cfa_paged_tables(cfa_paged *p, int n_seqs, int base, const int *lens, const int *fresh,
                            const int *free_pages, int n_free, const int *pool, int *tables,
                            int table_width, int *lens_out, int *pool_out, int *cu, int *positions,
                            int *slots, int n_slots, void *stream) {
    if (!p || n_seqs < 1 || n_seqs > p->max_seqs || base < 0 || !lens || !fresh || n_free < 0 ||
        (n_free > 0 && !free_pages) || !pool || !tables || table_width < 1 ||
        table_width > cfa::kPagedMaxTableWidth ||
        static_cast<long long>(table_width) * p->ps > (1 << 30) || base > (1 << 30) || !lens_out ||
        !pool_out || !cu || !positions || !slots || n_slots < 1 || n_slots > p->max_tokens)
        return fail(CFA_ERR_INVALID_ARG);
    const size_t B4 = 4u * static_cast<size_t>(n_seqs), S4 = 4u * static_cast<size_t>(n_slots);
    const struct { const void *at; size_t n; } in[] = {
        {lens, B4}, {fresh, B4}, {free_pages, 4u * static_cast<size_t>(n_free)}, {pool, 8}};
    const struct { const void *at; size_t n; const void *may; } outs[] = {
        {tables, B4 * table_width, nullptr}, {lens_out, B4, lens}, {pool_out, 8, pool},
        {cu, B4 + 4, nullptr}, {positions, S4, nullptr}, {slots, S4, nullptr}};
    for (const auto &i : in)
        if (!aligned(i.at, 4)) return fail(CFA_ERR_ALIGNMENT);
    for (int a = 0; a < 6; ++a) {
        if (!aligned(outs[a].at, 4)) return fail(CFA_ERR_ALIGNMENT);
        for (const auto &i : in)
            if (overlaps(outs[a].at, outs[a].n, i.at, i.n) && !(outs[a].may == i.at && outs[a].at == i.at))
                return fail(CFA_ERR_INVALID_ARG);
        for (int b = 0; b < a; ++b)
            if (overlaps(outs[a].at, outs[a].n, outs[b].at, outs[b].n)) return fail(CFA_ERR_INVALID_ARG);
    }
    OnDevice on(p->device);
    if (!on.ok()) return fail(CFA_ERR_CUDA);
    cfa::TablesParams kp{};
    kp.lens = lens;
    kp.fresh = fresh;
    kp.free_pages = free_pages;
    kp.pool = pool;
    kp.tables = tables;
    kp.lens_out = lens_out;
    kp.pool_out = pool_out;
    kp.cu = cu;
    kp.positions = positions;
    kp.slots = slots;
    kp.status = p->words;
    kp.ticket = p->words + 1;
    kp.B = n_seqs;
    kp.width = table_width;
    kp.page_size = p->ps;
    kp.n_free = n_free;
    kp.n_slots = n_slots;
    kp.base = base;
    kp.max_page = static_cast<int>(((1ll << 31) - 1) / p->ps) - 1;
    const int grid = std::min(p->num_sms, (n_slots + cfa::kTablesThreads - 1) / cfa::kTablesThreads);
    void *args[1] = {&kp};
    const cfa_status st = launch(cfa::paged_tables_kernel_ptr(), grid, cfa::kTablesThreads,
                                 sizeof(int) * (3u * static_cast<size_t>(n_seqs) + 2),
                                 static_cast<cudaStream_t>(stream), args);
    return st == CFA_OK ? CFA_OK : fail(st);
}

cfa_status cfa_paged_append(cfa_paged *p, int n_tokens, const void *q, long long q_stride,
                            const void *k, long long k_stride, const void *v, long long v_stride,
                            const int *positions, const int *slots, int n_pages, void *k_pages,
                            void *v_pages, void *q_out, void *stream) {
    if (!p) return fail(CFA_ERR_INVALID_ARG);
    const AppendArgs a{n_tokens, q, k, v, q_stride, k_stride, v_stride, positions, slots, n_pages,
                       k_pages, v_pages, q_out};
    cfa_status st = check_append(p, a);
    if (st != CFA_OK) return fail(st);
    OnDevice on(p->device);
    if (!on.ok()) return fail(CFA_ERR_CUDA);
    st = launch_append(p, a, static_cast<cudaStream_t>(stream));
    return st == CFA_OK ? CFA_OK : fail(st);
}

cfa_status cfa_paged_attention(cfa_paged *p, int n_tokens, int n_seqs, const void *q,
                               long long q_stride, const int *cu, const int *prefix_table,
                               int prefix_len, const int *tables, int table_width, const int *lens,
                               int n_pages, const void *k_pages, const void *v_pages, float scale,
                               void *out, float *lse, void *stream) {
    if (!p) return fail(CFA_ERR_INVALID_ARG);
    const AttnArgs a{n_tokens, n_seqs, q, q_stride, cu, prefix_table, prefix_len, tables,
                     table_width, lens, n_pages, k_pages, v_pages, scale, out, lse};
    cfa_status st = check_attention(p, a);
    if (st != CFA_OK) return fail(st);
    OnDevice on(p->device);
    if (!on.ok()) return fail(CFA_ERR_CUDA);
    st = launch_attention(p, a, static_cast<cudaStream_t>(stream));
    return st == CFA_OK ? CFA_OK : fail(st);
}

cfa_status cfa_paged_layer(cfa_paged *p, int n_tokens, int n_seqs, const void *q,
                           long long q_stride, const void *k, long long k_stride, const void *v,
                           long long v_stride, const int *positions, const int *slots,
                           const int *cu, const int *prefix_table, int prefix_len,
                           const int *tables, int table_width, const int *lens, int n_pages,
                           void *k_pages, void *v_pages, float scale, void *q_out, void *out,
                           float *lse, void *stream) {
    if (!p) return fail(CFA_ERR_INVALID_ARG);
    const AppendArgs a{n_tokens, q, k, v, q_stride, k_stride, v_stride, positions, slots, n_pages,
                       k_pages, v_pages, q_out};
    const AttnArgs b{n_tokens, n_seqs, q_out, static_cast<long long>(p->nh) * p->D, cu,
                     prefix_table, prefix_len, tables, table_width, lens, n_pages, k_pages, v_pages,
                     scale, out, lse};
    cfa_status st = check_layer(p, a, b);
    if (st != CFA_OK) return fail(st);
    OnDevice on(p->device);
    if (!on.ok()) return fail(CFA_ERR_CUDA);
    st = launch_append(p, a, static_cast<cudaStream_t>(stream));
    if (st == CFA_OK) st = launch_attention(p, b, static_cast<cudaStream_t>(stream));
    return st == CFA_OK ? CFA_OK : fail(st);
}

cfa_status cfa_paged_status(cfa_paged *p) {
    if (!p) return fail(CFA_ERR_INVALID_ARG);
    OnDevice on(p->device);
    unsigned v = 0;
    if (!on.ok() || cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(&v, p->words, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess ||
        !clear_words(p->words, 1)) {
        cudaGetLastError();
        return fail(CFA_ERR_CUDA);
    }
    if (v & cfa::kStatusTimeoutBit) return fail(CFA_ERR_TIMEOUT);
    if (v & (cfa::kStatusBadLengthBit | cfa::kStatusBadPageBit)) return fail(CFA_ERR_INVALID_ARG);
    if (v & cfa::kStatusNoPagesBit) return fail(CFA_ERR_NO_PAGES);
    return CFA_OK;
}

cfa_status cfa_paged_describe(const cfa_paged *p, char *buf, int len) {
    if (!p || !buf || len < 1) return fail(CFA_ERR_INVALID_ARG);
    std::snprintf(buf, static_cast<size_t>(len),
                  "{\"max_seqs\": %d, \"max_tokens\": %d, \"n_heads\": %d, \"n_kv_heads\": %d, "
                  "\"head_dim\": %d, \"page_size\": %d, \"rotary_dim\": %d, \"interleaved\": %d, "
                  "\"scaling\": %d, \"num_sms\": %d, \"smem_bytes\": %d, \"workspace_bytes\": %lld, "
                  "\"plan_bytes\": %lld}",
                  p->max_seqs, p->max_tokens, p->nh, p->nkv, p->D, p->ps, p->rd, p->interleaved,
                  p->scaling, p->num_sms, cfa::paged_attention_smem(p->D, p->max_seqs),
                  p->rec_rows * (4ll * p->D + 8), static_cast<long long>(sizeof(int) * p->plan_ints));
    return CFA_OK;
}

}  // extern "C"
