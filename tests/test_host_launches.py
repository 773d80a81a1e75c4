"""Host code of the launches, compiled on the CPU from its own source text (taken out
of the .cu files by brace matching) against stand-ins for the CUDA runtime that record what
they are asked.

- `selector_loss_launch`: the shared memory a kernel is allowed is the same whichever call
  asks for it, and covers every call of that kernel.  (The allowance belongs to the kernel,
  not to the call: were it a call's own, one host thread could lower it between another's
  asking and launching.)
- `allow_smem`, through which every other kernel asks: an allowance is never lowered, is each
  device's and each kernel's own, and a refused one leaves the last.
- `largest_cluster` of the sort: asked once a device, of each device for itself, and
  without memory from the C++ heap, whose exhaustion would leave the C entry as an
  exception.
"""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dflash2_draft_block_gb300", "csrc")


def _read(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _block(text, start):
    """From `start` (which must occur once) through its balanced closing brace and a ';'."""
    assert text.count(start) == 1, start
    i = text.index(start)
    depth = 0
    for k in range(text.index("{", i), len(text)):
        depth += (text[k] == "{") - (text[k] == "}")
        if text[k] == "}" and depth == 0:
            return text[i:k + 1] + (";" if text[k + 1:k + 2] == ";" else "")
    raise AssertionError("unbalanced braces after " + start)


def _line(text, start):
    assert text.count(start) == 1, start
    i = text.index(start)
    return text[i:text.index("\n", i)]


STUBS = r"""
#include <atomic>
#include <climits>
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <mutex>
#include <new>
#include <unordered_map>
#define __host__
#define __device__
#define __forceinline__ inline
#define DF2_MAX_TOPK 1024
#define DF2_MAX_RANK 4096
typedef int cudaError_t;
typedef void* cudaStream_t;
enum { cudaSuccess = 0, cudaErrorInvalidValue = 1 };
enum { cudaFuncAttributeMaxDynamicSharedMemorySize = 8, cudaFuncAttributeNonPortableClusterSizeAllowed = 14 };
enum { cudaLaunchAttributeProgrammaticStreamSerialization = 6, cudaLaunchAttributeClusterDimension = 4 };
struct dim3 { unsigned x, y, z; explicit dim3(unsigned a = 1) : x(a), y(1), z(1) {} };
struct cudaLaunchAttribute {
    int id;
    struct { int programmaticStreamSerializationAllowed; dim3 clusterDim; } val;
};
struct cudaLaunchConfig_t {
    dim3 gridDim, blockDim;
    size_t dynamicSmemBytes = 0;
    cudaStream_t stream = nullptr;
    cudaLaunchAttribute* attrs = nullptr;
    int numAttrs = 0;
};
template <class T> T dmin(T a, T b) { return a < b ? a : b; }
template <class T> T dmax(T a, T b) { return a < b ? b : a; }
void note_launch() {}
// memory runs out where a test says so; the device, and how many large clusters fit on it
bool g_no_memory;
int g_device, g_fit, g_asked;
cudaError_t cudaGetDevice(int* d) { *d = g_device; return cudaSuccess; }
template <class K> cudaError_t cudaOccupancyMaxActiveClusters(int* n, K*, const cudaLaunchConfig_t*) {
    ++g_asked;
    *n = g_fit;
    return cudaSuccess;
}
// the kernel last asked for or launched, and with how much
const void* g_kernel;
long long g_allowed, g_used;
template <class K> cudaError_t cudaFuncSetAttribute(K* k, int which, int value) {
    g_kernel = reinterpret_cast<const void*>(k);
    if (which != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
    if (value > 227 * 1024) return cudaErrorInvalidValue;
    g_allowed = value;
    return cudaSuccess;
}
template <class K, class... A> cudaError_t cudaLaunchKernelEx(const cudaLaunchConfig_t* c, K* k, A&&...) {
    g_kernel = reinterpret_cast<const void*>(k);
    g_used = (long long)c->dynamicSmemBytes;
    return cudaSuccess;
}
"""


def _loss_source():
    loss, kernels = _read("selector_loss.cu"), _read("kernels.h")
    return "\n".join([
        _block(kernels, "struct ZeroArgs {"),
        _line(loss, "constexpr int kMaxWarps"),
        _block(loss, "struct LossArgs {"),
        _line(loss, "constexpr int kZeroBytes"),
        _line(loss, "constexpr int kZeroBlocks"),
        _block(loss, "__host__ __device__ __forceinline__ int64_t zero_units("),
        _line(loss, "constexpr size_t loss_smem("),
        "template <int L, int CH> void selector_loss_kernel(const LossArgs, int) { g_used += L * 100 + CH; }",
        "template <int L, int CH>\n" + _block(loss, "cudaError_t launch(LossArgs a, int64_t P, cudaStream_t stream) {"),
        _block(loss, "cudaError_t selector_loss_launch("),
        r"""
extern "C" int loss_smem_of(int64_t P, int K, int r, int64_t cleared, long long* kernel, long long* allowed, long long* used) {
    ZeroArgs z{};
    z.bytes[0] = cleared;
    g_kernel = nullptr;
    g_allowed = -1;
    const int rc = selector_loss_launch(nullptr, nullptr, P, nullptr, nullptr, nullptr, nullptr, nullptr, 1 << 20, K, r, nullptr,
                                        nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, z, nullptr, false, nullptr);
    *kernel = (long long)(intptr_t)g_kernel;
    *allowed = g_allowed;
    *used = g_used;
    return rc;
}
"""])


def _sort_source():
    sort = _read("token_sort.cu")
    return "\n".join([
        "void* operator new(size_t n) { if (g_no_memory) throw std::bad_alloc(); return malloc(n ? n : 1); }",
        "void operator delete(void* p) noexcept { free(p); }",
        "void operator delete(void* p, size_t) noexcept { free(p); }",
        "struct SortArgs {};",
        "template <int ITEMS> void token_sort_kernel(const SortArgs) {}",
        "template <int ITEMS> size_t sort_smem(int bins) { return bins * ITEMS; }",
        _line(sort, "constexpr int kMaxCluster"),
        _line(sort, "constexpr int kMaxDigitBits"),
        _line(sort, "constexpr int kMaxBins"),
        "".join(_line(sort, k) + "\n" for k in ("constexpr int kMaxDevices",) if k in sort),
        "template <int ITEMS>\n" + _block(sort, "cudaError_t largest_cluster(cudaLaunchConfig_t* cfg, int* most) {"),
        r"""
extern "C" int cluster_of(int device, int fit, int no_memory, int* most, int* asked) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg;
    cfg.attrs = attr;
    g_device = device;
    g_fit = fit;
    g_asked = 0;
    g_no_memory = no_memory != 0;
    int rc;
    try {
        rc = largest_cluster<2>(&cfg, most);
    } catch (...) {
        rc = -1;
    }
    g_no_memory = false;
    *asked = g_asked;
    return rc;
}
"""])


def _allow_source():
    return "template <auto Kernel>\n" + _block(_read("common.cuh"), "cudaError_t allow_smem(size_t bytes) {") + r"""
void first_kernel(int) { g_used = 1; }
void second_kernel(int) { g_used = 2; }
extern "C" long long allowed(int second, int device, long long bytes) {
    g_device = device;
    g_allowed = -1;
    const int rc = second ? allow_smem<second_kernel>(size_t(bytes)) : allow_smem<first_kernel>(size_t(bytes));
    return rc == cudaSuccess ? g_allowed : -1;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("host_training")
    src, lib = d / "host.cpp", d / "host.so"
    src.write_text(STUBS + _loss_source() + _sort_source() + _allow_source())
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-o", str(lib), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(lib))


def test_a_kernel_s_shared_memory_does_not_depend_on_the_call(host):
    allowances, largest = {}, {}
    k, a, u = (ctypes.c_longlong() for _ in range(3))
    for r in (8, 32, 40, 64, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 1536, 2048, 2056, 2064, 3000 // 8 * 8, 4088, 4096):
        for K in (1, 7, 16, 33, 64, 129, 500, 1024):
            for P in (1, 40, 607, 608, 5000):
                for cleared in (0, 1 << 20):
                    assert host.loss_smem_of(ctypes.c_int64(P), K, r, ctypes.c_int64(cleared), ctypes.byref(k),
                                             ctypes.byref(a), ctypes.byref(u)) == 0
                    largest[k.value] = max(largest.get(k.value, 0), u.value)
                    if a.value >= 0:
                        allowances.setdefault(k.value, set()).add(a.value)
                    else:
                        assert u.value <= 48 * 1024       # what a kernel may use unasked
    assert allowances and len(largest) == 8
    for kernel, values in allowances.items():
        assert len(values) == 1, f"{len(values)} allowances, {min(values)} .. {max(values)}"
        assert largest[kernel] <= max(values) <= 227 * 1024


def test_an_allowance_is_never_lowered(host):
    host.allowed.restype = ctypes.c_longlong
    ask = lambda second, device, bytes_: host.allowed(second, device, ctypes.c_longlong(bytes_))
    assert ask(0, 0, 100_000) == 100_000 and ask(0, 0, 50_000) == 100_000
    assert ask(0, 0, 227 * 1024 + 1) == -1 and ask(0, 0, 1) == 100_000
    assert ask(0, 0, 150_000) == 150_000 and ask(0, 0, 100_000) == 150_000
    assert ask(0, 3, 60_000) == 60_000 and ask(1, 0, 70_000) == 70_000
    assert ask(0, 64, 80_000) == 80_000
    # and nobody asks in another way, but for what does not depend on the call
    for name in sorted(os.listdir(CSRC)):
        if name not in ("common.cuh", "selector_loss.cu", "token_sort.cu"):
            assert "cudaFuncAttributeMaxDynamicSharedMemorySize" not in _read(name), name


def test_the_largest_cluster_of_each_device(host):
    most, asked = ctypes.c_int(), ctypes.c_int()

    def ask(device, fit, no_memory=0):
        assert host.cluster_of(device, fit, no_memory, ctypes.byref(most), ctypes.byref(asked)) == 0
        return most.value, asked.value

    assert ask(0, 3, no_memory=1) == (16, 1)
    assert ask(0, 0) == (16, 0)                  # known
    assert ask(5, 0, no_memory=1) == (8, 1)      # no such cluster fits: the portable size
    assert ask(5, 0) == (8, 0) and ask(0, 0) == (16, 0)
    for device in (63, 64, 1000):                # past any table of devices as well
        assert ask(device, 2, no_memory=1)[0] == 16
