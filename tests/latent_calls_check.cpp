// Checks of the latent-cache entry points' host code with a stand-in for the CUDA runtime that
// writes down what is called: which calls are refused, which kernels a call launches, and in which order
// the device's work is asked for. The argument names the check. Prints "ok" or what is wrong.
#include "cfa_latent.cu"

#include <cstdlib>
#include <string>
#include <vector>

namespace {
std::vector<std::string> calls;
cudaError_t note(const char *what) {
    calls.push_back(what);
    return cudaSuccess;
}
size_t allocated;
char kernels[10];
struct Map {
    const void *base;
    uint64_t cols, rows, stride;
    uint32_t box_cols, box_rows;
};
std::vector<Map> maps;
dim3 grid;
}  // namespace

extern "C" {
cudaError_t CUDARTAPI cudaGetDevice(int *d) { return *d = 0, cudaSuccess; }
cudaError_t CUDARTAPI cudaSetDevice(int) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaGetLastError(void) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaMalloc(void **p, size_t n) { return allocated += n, *p = std::malloc(64), cudaSuccess; }
cudaError_t CUDARTAPI cudaFree(void *p) { return std::free(p), cudaSuccess; }
cudaError_t CUDARTAPI cudaMemset(void *, int, size_t) { return note("set"); }
cudaError_t CUDARTAPI cudaMemcpy(void *to, const void *, size_t n, cudaMemcpyKind) { return std::memset(to, 0, n), note("copy"); }
cudaError_t CUDARTAPI cudaStreamSynchronize(cudaStream_t) { return note("wait"); }
cudaError_t CUDARTAPI cudaDeviceSynchronize(void) { return note("wait"); }
cudaError_t CUDARTAPI cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *kernel, void **) {
    static const char *names[] = {"append", "fold", "unfold", "fold tcgen05", "unfold tcgen05", "attention", "merge", "expanded", "expanded merge"};
    grid = c->gridDim;
    return note(names[static_cast<const char *>(kernel) - kernels]);
}
}

namespace cfa {
const void *latent_append_kernel_ptr(bool) { return kernels; }
const void *latent_heads_kernel_ptr(bool fold) { return kernels + (fold ? 1 : 2); }
int latent_heads_smem(bool) { return 1 << 15; }
const void *latent_heads_mma_kernel_ptr(bool fold) { return kernels + (fold ? 3 : 4); }
int latent_heads_mma_smem(bool) { return 1 << 17; }
const void *latent_attention_kernel_ptr() { return kernels + 5; }
const void *latent_merge_kernel_ptr() { return kernels + 6; }
const void *latent_expanded_kernel_ptr() { return kernels + 7; }
const void *latent_expanded_merge_kernel_ptr() { return kernels + 8; }
int latent_attention_smem() { return 1 << 17; }
int latent_expanded_smem() { return 1 << 17; }
cfa_status encode_bf16_2d_ex(CUtensorMap *, const void *base, uint64_t cols, uint64_t rows, uint64_t stride, uint32_t bc, uint32_t br,
                             bool) {
    maps.push_back({base, cols, rows, stride, bc, br});
    return CFA_OK;
}
cfa_status set_last_error(cfa_status s) { return s; }
}  // namespace cfa

namespace {

using Calls = std::vector<std::string>;

// Calls whose arrays lie apart, at addresses that nobody reads.
struct Args {
    static constexpr int T = 8, B = 3, H = 4, PS = 16, PAGES = 4, W = 2, S = 20;
    uintptr_t a = 0x1000000, g = 0x1800000, q = 0x2000000, pos = 0x3000000, slots = 0x4000000, cu = 0x5000000, tables = 0x6000000,
              lens = 0x7000000, pages = 0x8000000, w = 0x9000000, q_out = 0xa000000, q_lat = 0xb000000, o_lat = 0xc000000,
              lse = 0xd000000, out = 0xe000000, kv = 0xf000000, rope = 0x11000000, cu_k = 0x12000000;
    static const int *ints(uintptr_t x) { return reinterpret_cast<const int *>(x); }
    static void *at(uintptr_t x) { return reinterpret_cast<void *>(x); }
    cfa_status layer(cfa_latent *p, float scale = 0.f, float eps = 1e-6f) const {
        return cfa_latent_layer(p, T, B, at(a), 640, at(g), eps, at(q), H * 192, ints(pos), ints(slots), ints(cu), ints(tables), W,
                                ints(lens), PAGES, at(pages), at(w), scale, at(q_out), at(q_lat), at(o_lat),
                                static_cast<float *>(at(lse)), at(out), nullptr);
    }
    cfa_status expanded(cfa_latent *p, int keys = S, long long qs = H * 192, long long kvs = H * 256 + 8, long long rs = 576) const {
        return cfa_latent_expanded(p, T, keys, B, at(q), qs, at(kv), kvs, at(rope), rs, ints(cu), ints(cu_k), 0.f, at(out),
                                   static_cast<float *>(at(lse)), nullptr);
    }
};

cfa_latent *plan() { return cfa_latent_create(Args::B, Args::T, Args::H, Args::PS); }

// What a call writes lies apart from everything else that it, or a later part of it, touches.
const char *overlaps() {
    cfa_latent *p = plan();
    if (!p) return "no plan";
    using M = uintptr_t Args::*;
    constexpr uintptr_t T = Args::T, H = Args::H, B = Args::B;
    struct Array {
        M at;
        uintptr_t bytes;
    };
    const Array written[] = {{&Args::pages, 2 * Args::PAGES * Args::PS * 576}, {&Args::q_out, 2 * T * H * 192},
                             {&Args::q_lat, 2 * T * H * 576}, {&Args::o_lat, 2 * T * H * 512}, {&Args::lse, 4 * T * H},
                             {&Args::out, 2 * T * H * 128}};
    const Array read[] = {{&Args::a, 2 * ((T - 1) * 640 + 576)}, {&Args::g, 1024}, {&Args::q, 2 * T * H * 192}, {&Args::pos, 4 * T},
                          {&Args::slots, 4 * T}, {&Args::cu, 4 * (B + 1)}, {&Args::tables, 4 * B * Args::W}, {&Args::lens, 4 * B},
                          {&Args::w, 2 * 512 * 256 * H}};
    calls.clear();
    if (Args{}.layer(p) != CFA_OK || calls != Calls{"append", "fold", "attention", "merge", "unfold"}) return "a good layer was refused";
    Args same;
    same.q_out = same.q;
    if (same.layer(p) != CFA_OK) return "rotation in place was refused";
    auto tried = [&](const Array &w, const Array &r) -> const char * {
        for (const uintptr_t off : {uintptr_t(16), w.bytes - 16, (w.bytes + 15) & ~uintptr_t(15), uintptr_t(0) - ((r.bytes + 15) & ~uintptr_t(15))}) {
            Args c;
            c.*r.at = c.*w.at + off;
            const bool apart = off != 16 && off != w.bytes - 16;
            calls.clear();
            const cfa_status st = c.layer(p);
            if (apart ? st != CFA_OK : st != CFA_ERR_INVALID_ARG) return apart ? "arrays side by side were refused" : "an overlap was taken";
            if (!apart && !calls.empty()) return "a refused call launched";
        }
        return nullptr;
    };
    for (const Array &w : written) {
        for (const Array &r : read)
            if (const char *wrong = tried(w, r)) return wrong;
        for (const Array &v : written)
            if (v.at != w.at)
                if (const char *wrong = tried(w, v)) return wrong;
    }
    // the expanded form
    const Array results[] = {{&Args::out, 2 * T * H * 128}, {&Args::lse, 4 * T * H}};
    const Array inputs[] = {{&Args::q, 2 * T * H * 192}, {&Args::kv, 2 * ((Args::S - 1) * (H * 256 + 8) + H * 256)},
                            {&Args::rope, 2 * ((Args::S - 1) * 576 + 64)}, {&Args::cu, 4 * (B + 1)}, {&Args::cu_k, 4 * (B + 1)}};
    calls.clear();
    if (Args{}.expanded(p) != CFA_OK || calls != Calls{"expanded", "expanded merge"}) return "a good prompt was refused";
    for (const Array &w : results)
        for (const Array &r : inputs)
            for (const uintptr_t off : {uintptr_t(16), uintptr_t(0) - r.bytes / 16 * 16 + 16}) {
                Args c;
                c.*r.at = c.*w.at + off;
                if (c.expanded(p) != CFA_ERR_INVALID_ARG) return "the expanded form took an overlap";
            }
    cfa_latent_destroy(p);
    return nullptr;
}

// Arguments out of their ranges.
const char *ranges() {
    cfa_latent *p = plan();
    if (!p) return "no plan";
    const Args c;
    auto at = [](uintptr_t x) { return Args::at(x); };
    constexpr int T = Args::T, H = Args::H;
    for (const float bad : {-1.f, 2.4e38f, 3.4e38f, HUGE_VALF, NAN})
        if (c.layer(p, bad) != CFA_ERR_INVALID_ARG) return "a scale was taken";
    for (const float good : {0.f, 1e-45f, 0.0721f, 2.3e38f})
        if (c.layer(p, good) != CFA_OK) return "a scale was refused";
    for (const float bad : {-1e-9f, HUGE_VALF, NAN})
        if (c.layer(p, 0.f, bad) != CFA_ERR_INVALID_ARG) return "an eps was taken";
    if (c.layer(p, 0.f, 0.f) != CFA_OK) return "eps 0 was refused";
    if (cfa_latent_fold(p, T + 1, at(c.q), H * 192, at(c.w), at(c.q_lat), nullptr) != CFA_ERR_INVALID_ARG) return "too many tokens";
    if (cfa_latent_fold(p, -1, at(c.q), H * 192, at(c.w), at(c.q_lat), nullptr) != CFA_ERR_INVALID_ARG) return "fewer than no tokens";
    for (const long long bad : {0ll, H * 192ll - 8, H * 192ll + 4, 1ll << 36})
        if (cfa_latent_fold(p, T, at(c.q), bad, at(c.w), at(c.q_lat), nullptr) != CFA_ERR_INVALID_ARG) return "a stride was taken";
    if (cfa_latent_fold(p, T, at(c.q + 8), H * 192, at(c.w), at(c.q_lat), nullptr) != CFA_ERR_ALIGNMENT) return "8 bytes were enough";
    if (cfa_latent_unfold(p, T, at(c.o_lat), at(c.w + 8), at(c.out), nullptr) != CFA_ERR_ALIGNMENT) return "8 bytes were enough";
    if (cfa_latent_unfold(p, T, at(c.o_lat), nullptr, at(c.out), nullptr) != CFA_ERR_INVALID_ARG) return "no weights";
    if (c.expanded(p, -1) != CFA_ERR_INVALID_ARG || c.expanded(p, (1 << 30) + 1) != CFA_ERR_INVALID_ARG) return "a number of keys was taken";
    if (c.expanded(p, Args::S, H * 192, H * 256 - 8) != CFA_ERR_INVALID_ARG || c.expanded(p, Args::S, H * 192, H * 256, 56) != CFA_ERR_INVALID_ARG)
        return "a key stride was taken";
    // without keys there is nothing to point at
    if (cfa_latent_expanded(p, T, 0, 1, at(c.q), H * 192, nullptr, 0, nullptr, 0, Args::ints(c.cu), Args::ints(c.cu_k), 0.f, at(c.out),
                            nullptr, nullptr) != CFA_OK)
        return "no keys were refused";
    // no tokens: no pointers, no launch
    calls.clear();
    if (cfa_latent_append(p, 0, nullptr, 0, nullptr, 0.f, nullptr, 0, nullptr, nullptr, 0, nullptr, nullptr, nullptr) != CFA_OK ||
        cfa_latent_fold(p, 0, nullptr, 0, nullptr, nullptr, nullptr) != CFA_OK ||
        cfa_latent_unfold(p, 0, nullptr, nullptr, nullptr, nullptr) != CFA_OK ||
        cfa_latent_attention(p, 0, 0, nullptr, nullptr, nullptr, 0, nullptr, 0, nullptr, 0.f, nullptr, nullptr, nullptr) != CFA_OK ||
        cfa_latent_expanded(p, 0, 0, 0, nullptr, 0, nullptr, 0, nullptr, 0, nullptr, nullptr, 0.f, nullptr, nullptr, nullptr) != CFA_OK ||
        !calls.empty())
        return "no tokens";
    // tables and pages
    auto attend = [&](int seqs, int width, int pages) {
        return cfa_latent_attention(p, T, seqs, at(c.q_lat), Args::ints(c.cu), Args::ints(c.tables), width, Args::ints(c.lens), pages,
                                    at(c.pages), 0.f, at(c.o_lat), nullptr, nullptr);
    };
    if (attend(0, 2, 4) != CFA_ERR_INVALID_ARG || attend(Args::B + 1, 2, 4) != CFA_ERR_INVALID_ARG) return "a number of requests was taken";
    if (attend(1, 0, 4) != CFA_ERR_INVALID_ARG || attend(1, (1 << 18) + 1, 4) != CFA_ERR_INVALID_ARG) return "a table width was taken";
    if (attend(1, 2, 0) != CFA_ERR_INVALID_ARG || attend(1, 2, 1 << 27) != CFA_ERR_INVALID_ARG) return "a number of pages was taken";
    if (cfa_latent_set_rope(p, 0.5, 0, 0, 1, 1, 32, 4096, 1) != CFA_ERR_INVALID_ARG || cfa_latent_set_rope(p, 1e4, 0, 3, 1, 1, 32, 4096, 1) != CFA_ERR_INVALID_ARG ||
        cfa_latent_set_rope(p, 1e4, 0, 2, 4, 32, 1, 4096, 1) != CFA_ERR_INVALID_ARG || cfa_latent_set_rope(p, 0.0, 1, 9, -1, 0, 0, 0, -1) != CFA_OK)
        return "rotations";
    cfa_latent_destroy(p);
    return nullptr;
}

// Words are cleared before create and status return, as kernels on other streams do not wait for a memset.
const char *order() {
    calls.clear();
    cfa_latent *p = plan();
    if (!p) return "no plan";
    if (calls != Calls{"set", "wait"}) return "create leaves its words to be cleared later";
    calls.clear();
    if (cfa_latent_status(p) != CFA_OK) return "status";
    if (calls != Calls{"wait", "copy", "set", "wait"}) return "status leaves its word to be cleared later";
    cfa_latent_destroy(p);
    return nullptr;
}

// describe tells of every byte that a plan keeps on the device (and four words).
const char *bytes() {
    for (const int heads : {1, 128}) {
        allocated = 0;
        cfa_latent *p = cfa_latent_create(64, 512, heads, 64);
        char text[1024];
        if (!p || cfa_latent_describe(p, text, sizeof text) != CFA_OK) return "no plan";
        const char *name = "\"workspace_bytes\": ", *at = std::strstr(text, name);
        if (!at) return "a field is missing";
        if (std::atoll(at + std::strlen(name)) + 16 != static_cast<long long>(allocated)) return "bytes that describe leaves out";
        cfa_latent_destroy(p);
    }
    return nullptr;
}

// Which form of the folding products a call takes, and the boxes that its copies are made of: inside a page, and no
// larger than what is there.
const char *forms() {
    const struct {
        int T, H;
        bool fold, many;
    } cases[] = {{1, 128, true, false}, {48, 128, true, false}, {49, 128, true, true}, {192, 32, true, false}, {193, 32, true, true},
                 {1, 128, false, false}, {16, 128, false, false}, {17, 128, false, true}, {80, 32, false, false}, {81, 32, false, true}};
    for (const auto &c : cases) {
        cfa_latent *p = cfa_latent_create(4, 4096, c.H, 64);
        const Args a;
        calls.clear();
        maps.clear();
        const cfa_status st = c.fold ? cfa_latent_fold(p, c.T, Args::at(a.q), c.H * 192, Args::at(1ull << 40), Args::at(1ull << 41), nullptr)
                                     : cfa_latent_unfold(p, c.T, Args::at(a.q), Args::at(1ull << 40), Args::at(1ull << 41), nullptr);
        const std::string want = std::string(c.fold ? "fold" : "unfold") + (c.many ? " tcgen05" : "");
        if (st != CFA_OK || calls != Calls{want}) return "another form than its rule says";
        if (c.many && (maps.size() != 3 || maps[0].rows != static_cast<uint64_t>(c.T) || maps[2].rows != static_cast<uint64_t>(c.T)))
            return "maps past the last token";
        cfa_latent_destroy(p);
    }
    for (const int ps : {16, 32, 64, 128, 192}) {
        cfa_latent *p = cfa_latent_create(4, 64, 8, ps);
        maps.clear();
        const Args a;
        if (cfa_latent_attention(p, 2, 1, Args::at(a.q_lat), Args::ints(a.cu), Args::ints(a.tables), 2, Args::ints(a.lens), 3, Args::at(a.pages),
                                 0.f, Args::at(a.o_lat), nullptr, nullptr) != CFA_OK ||
            maps.size() != 2)
            return "a good call was refused";
        if (maps[0].rows != 16 || maps[1].rows != static_cast<uint64_t>(3 * ps) || ps % maps[1].box_rows || 64 % maps[1].box_rows) return "boxes";
        cfa_latent_destroy(p);
    }
    return nullptr;
}

}  // namespace

int main(int argc, char **argv) {
    const std::string which = argc > 1 ? argv[1] : "";
    const char *wrong = which == "overlaps" ? overlaps()
                        : which == "ranges" ? ranges()
                        : which == "order"  ? order()
                        : which == "bytes"  ? bytes()
                        : which == "forms"  ? forms()
                                            : "which check?";
    std::puts(wrong ? wrong : "ok");
    return wrong != nullptr;
}
