// Checks of the paged-cache entry points' host code with a stand-in for the CUDA runtime that
// writes down what is called: which calls are refused, and in which order the device's work is
// asked for. The argument names the check. Prints "ok" or what is wrong.
#include "cfa_paged.cu"

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
cfa::PagedAttnParams merged;
char kernels[4];
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
cudaError_t CUDARTAPI cudaMemcpy(void *to, const void *, size_t n, cudaMemcpyKind) {
    return std::memset(to, 0, n), note("copy");
}
cudaError_t CUDARTAPI cudaStreamSynchronize(cudaStream_t) { return note("wait"); }
cudaError_t CUDARTAPI cudaDeviceSynchronize(void) { return note("wait"); }
cudaError_t CUDARTAPI cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *kernel, void **args) {
    if (kernel == kernels + 3) merged = *static_cast<const cfa::PagedAttnParams *>(args[0]);
    return note("launch");
}
}

namespace cfa {
const void *paged_tables_kernel_ptr() { return kernels; }
const void *paged_append_kernel_ptr(bool) { return kernels + 1; }
const void *paged_attention_kernel_ptr(int) { return kernels + 2; }
const void *paged_merge_kernel_ptr(int) { return kernels + 3; }
int paged_attention_smem(int, int) { return 1 << 17; }
cfa_status encode_bf16_2d_ex(CUtensorMap *, const void *, uint64_t, uint64_t, uint64_t, uint32_t, uint32_t, bool) {
    return CFA_OK;
}
cfa_status set_last_error(cfa_status s) { return s; }
}  // namespace cfa

namespace {

// A layer call whose arrays lie apart, at addresses that nobody reads.
struct Layer {
    static constexpr int T = 8, B = 3, H = 4, KV = 2, D = 64, PS = 16, PAGES = 4, W = 2, P = 20;
    uintptr_t q = 0x1000000, k = 0x2000000, v = 0x3000000, pos = 0x4000000, slots = 0x5000000, cu = 0x6000000,
              prefix = 0x7000000, tables = 0x8000000, lens = 0x9000000, kp = 0xa000000, vp = 0xb000000,
              q_out = 0xc000000, out = 0xd000000, lse = 0xe000000;
    static const int *ints(uintptr_t a) { return reinterpret_cast<const int *>(a); }
    static void *at(uintptr_t a) { return reinterpret_cast<void *>(a); }
    cfa_status operator()(cfa_paged *p, float scale = 0.f) const {
        return cfa_paged_layer(p, T, B, at(q), H * D, at(k), KV * D, at(v), KV * D, ints(pos), ints(slots), ints(cu),
                               ints(prefix), P, ints(tables), W, ints(lens), PAGES, at(kp), at(vp), scale, at(q_out),
                               at(out), static_cast<float *>(at(lse)), nullptr);
    }
};

// What the append writes must not be what the attention reads its offsets and tables from.
const char *overlaps() {
    cfa_paged *p = cfa_paged_create(Layer::B, Layer::T, Layer::H, Layer::KV, Layer::D, Layer::PS);
    if (!p) return "no plan";
    const uintptr_t pages = 2 * Layer::PAGES * Layer::KV * Layer::PS * Layer::D, turned = 2 * Layer::T * Layer::H * Layer::D;
    calls.clear();
    if (Layer{}(p) != CFA_OK || calls != std::vector<std::string>(3, "launch")) return "a good call was refused";
    Layer in_place;
    in_place.q_out = in_place.q;
    if (in_place(p) != CFA_OK) return "rotation in place was refused";
    calls.clear();
    struct { uintptr_t Layer::*array; uintptr_t bytes; } read[] = {
        {&Layer::cu, 4 * (Layer::B + 1)}, {&Layer::lens, 4 * Layer::B}, {&Layer::tables, 4 * Layer::B * Layer::W},
        {&Layer::prefix, 4 * ((Layer::P + Layer::PS - 1) / Layer::PS)}, {&Layer::pos, 4 * Layer::T}, {&Layer::slots, 4 * Layer::T}};
    struct { uintptr_t Layer::*array; uintptr_t bytes; } written[] = {
        {&Layer::kp, pages}, {&Layer::vp, pages}, {&Layer::q_out, turned}, {&Layer::out, turned}, {&Layer::lse, 4 * Layer::T * Layer::H}};
    for (const auto &r : read)
        for (const auto &w : written)
            for (const uintptr_t off : {uintptr_t(0), w.bytes - 4, w.bytes, uintptr_t(0) - r.bytes, uintptr_t(4) - r.bytes}) {
                Layer c;
                c.*r.array = c.*w.array + off;
                const bool apart = off == w.bytes || off == uintptr_t(0) - r.bytes;
                const cfa_status st = c(p);
                if (apart ? st != CFA_OK : st != CFA_ERR_INVALID_ARG) return apart ? "arrays side by side were refused" : "an overlap was taken";
                if (!apart && !calls.empty()) return "a refused call launched";
                calls.clear();
            }
    cfa_paged_destroy(p);
    return nullptr;
}

// A memset runs in the legacy stream after the call that asks for it has returned, and a kernel
// on a stream that does not wait for that one may come first: the plan's words are cleared
// before create and status return.
const char *order() {
    using Calls = std::vector<std::string>;
    calls.clear();
    cfa_paged *p = cfa_paged_create(Layer::B, Layer::T, Layer::H, Layer::KV, Layer::D, Layer::PS);
    if (!p) return "no plan";
    if (calls != Calls{"set", "wait"}) return "create leaves its words to be cleared later";
    calls.clear();
    if (cfa_paged_status(p) != CFA_OK) return "status";
    if (calls != Calls{"wait", "copy", "set", "wait"}) return "status leaves its word to be cleared later";
    calls.clear();
    cfa_paged_destroy(p);
    return nullptr;
}

// A scale counts in 32 bits and times log2 e: neither may become infinite on the way.
const char *scales() {
    cfa_paged *p = cfa_paged_create(Layer::B, Layer::T, Layer::H, Layer::KV, Layer::D, Layer::PS);
    if (!p) return "no plan";
    for (const float good : {0.f, 1e-45f, 1e-38f, 0.125f, 1e10f, 2.3e38f})
        if (Layer{}(p, good) != CFA_OK) return "a scale was refused";
    for (const float bad : {-1.f, 2.4e38f, 3.4e38f, HUGE_VALF, NAN})
        if (Layer{}(p, bad) != CFA_ERR_INVALID_ARG) return "a scale was taken";
    cfa_paged_destroy(p);
    return nullptr;
}

// describe tells of every byte that a plan keeps on the device (and four words).
const char *bytes() {
    const struct { int seqs, tokens, heads, kv, d; } plans[] = {
        {1, 1, 1, 1, 64}, {2, 8, 4, 2, 64}, {64, 512, 32, 8, 128}, {1024, 1 << 17, 32, 32, 128}, {1024, 1 << 17, 1024, 1, 64}};
    for (const auto &s : plans) {
        allocated = 0;
        cfa_paged *p = cfa_paged_create(s.seqs, s.tokens, s.heads, s.kv, s.d, 64);
        char text[1024];
        if (!p || cfa_paged_describe(p, text, sizeof text) != CFA_OK) return "no plan";
        long long told = 0;
        for (const char *name : {"\"workspace_bytes\": ", "\"plan_bytes\": "}) {
            const char *at = std::strstr(text, name);
            if (!at) return "a field is missing";
            told += std::atoll(at + std::strlen(name));
        }
        if (told + 16 != static_cast<long long>(allocated)) return "bytes that describe leaves out";
        cfa_paged_destroy(p);
    }
    return nullptr;
}

// The clocks of a block's bytes are those that its head_dim's comment derives.
const char *clocks() {
    for (const int d : {64, 128}) {
        cfa_paged *p = cfa_paged_create(Layer::B, Layer::T, Layer::H, Layer::KV, d, Layer::PS);
        const Layer a;
        if (cfa_paged_attention(p, 1, 1, Layer::at(a.q), Layer::H * d, Layer::ints(a.cu), nullptr, 0, Layer::ints(a.tables),
                                1, Layer::ints(a.lens), 1, Layer::at(a.kp), Layer::at(a.vp), 0.f, Layer::at(a.out), nullptr,
                                nullptr) != CFA_OK)
            return "a good call was refused";
        const double clk = 512.0 * d * 152 / 6.8e12 * 1.9e9;
        const double unit = d == 128 ? 400 : 1350.0 / cfa::paged_cost(1);
        if (merged.block_clocks != std::lround(clk / unit)) return "other clocks than derived";
        cfa_paged_destroy(p);
    }
    return nullptr;
}

}  // namespace

int main(int argc, char **argv) {
    const std::string which = argc > 1 ? argv[1] : "";
    const char *wrong = which == "overlaps" ? overlaps() : which == "order" ? order() : which == "scales" ? scales() : which == "bytes" ? bytes() : which == "clocks" ? clocks() : "which check?";
    std::puts(wrong ? wrong : "ok");
    return wrong != nullptr;
}
