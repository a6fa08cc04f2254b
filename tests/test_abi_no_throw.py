"""No C++ exception leaves a C entry: a caller whose memory is exhausted gets the refusal of a bad
argument and its message like any other."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include "gdn_layer.h"

static bool exhausted = false;
void *operator new(std::size_t n) {
    if (exhausted) throw std::bad_alloc();
    return std::malloc(n);
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }

static int refused(gdn_status st, const char *word) {
    return st == GDN_ERR_INVALID_ARG && std::strstr(gdn_last_error(), word) != nullptr;
}

int main() {
    exhausted = true;
    gdn_linrec_step_args step = {};
    step.N = -5, step.D = 123456789;
    if (!refused(gdn_linrec_step(&step, nullptr), "bad sizes N=-5 D=123456789")) return 1;
    gdn_rms_norm_fwd_args norm = {};
    norm.rows = 3, norm.D = 64;
    if (!refused(gdn_rms_norm_fwd(&norm, nullptr), "sum (with a residual) are required")) return 2;
    gdn_mx_linear_args lin = {};
    if (gdn_mx_linear_workspace_size(&lin) < 256) return 3;
    lin.M = -1;
    if (gdn_mx_linear_workspace_size(&lin) != 0 || !std::strstr(gdn_last_error(), "null args or bad sizes")) return 4;
    std::puts("ok");
    return 0;
}
"""


def test_refusals_of_a_caller_without_memory(tmp_path):
    import __graft_entry__
    __graft_entry__.build()
    lib = os.path.join(ROOT, "gated_deltanet_linear_bwd_gb300")
    src, exe = tmp_path / "p.cpp", tmp_path / "p"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
                    os.path.join(lib, "libgdn.so"), f"-Wl,-rpath,{lib}"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert (r.returncode, r.stdout) == (0, "ok\n"), (r.returncode, r.stderr)
