"""No C++ exception leaves a C entry point when memory for its message runs out: a program whose
operator new throws calls each with an argument that it refuses."""
import subprocess

import pytest

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <dlfcn.h>
#include <new>
static bool fails = false;
void* operator new(std::size_t n)
{
    if (fails) throw std::bad_alloc();
    return std::malloc(n);
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

template <typename R, typename... A>
void call(void* lib, const char* name, A... args)
{
    auto f = reinterpret_cast<R (*)(A...)>(dlsym(lib, name));
    if (!f) std::exit(3);
    const char* what = "returned";
    fails = true;
    try {
        f(args...);
    } catch (...) {
        what = "threw";
    }
    fails = false;
    std::printf("%s %s\n", name, what);
}

int main(int, char** argv)
{
    void* lib = dlopen(argv[1], RTLD_NOW);
    if (!lib) {
        std::printf("%s\n", dlerror());
        return 2;
    }
    void* none = nullptr;
    const int64_t one = 1;
    call<int64_t>(lib, "gemm_rms_norm_grad_workspace", one, int64_t(7));
    call<int>(lib, "gemm_rms_norm", one, int64_t(7), none, none, none, 0.0f, none, none, 0, none,
              none, none);
    call<int>(lib, "gemm_mx_sizes", int64_t(-1), one, 0, none, none);
    call<int>(lib, "gemm_mx_quantize", one, int64_t(7), 0, 0, none, none, none, none, none, none);
    call<void*>(lib, "gemm_mx_create_plan", int64_t(0), one, one, 0, 0);
    call<void*>(lib, "gemm_mx_create_plan_beside", none, one, one, one, 0, 0, 0);
    call<int>(lib, "gemm_mx_set_wait", none, 0, 0);
    call<void*>(lib, "gemm_clip_create_plan", int64_t(-1), none, none, none, none);
    call<int>(lib, "gemm_clip_norm", none, none, none, none);
}
"""


@pytest.fixture(scope="module")
def b():
    from tma_pipelined_tensor_fp16_gb300 import binding, build
    build.build()
    return binding


def test_nothing_is_thrown(b, tmp_path):
    src, exe = tmp_path / "program.cpp", tmp_path / "program"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-rdynamic", str(src), "-o", str(exe), "-ldl"], check=True)
    out = subprocess.run([str(exe), b.LIB_PATH], check=True, capture_output=True, text=True).stdout
    lines = out.splitlines()
    assert len(lines) == 9 and not [line for line in lines if line.endswith("threw")], out
