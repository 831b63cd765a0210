"""The choice of a form for the 4-bit products, over all sizes that the entry point takes, on the host."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_sparse_attention_step_gb300",
                    "csrc")
X_BYTES = 128 * 1024


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text(f'#include "{CSRC}/matvec_plan.h"\n'
                   "using namespace csa2::mv::tc;\n"
                   'extern "C" long long x_of(long long n_kb, int C, int tok) { return x_bytes(n_kb, C, tok); }\n'
                   'extern "C" int plan_of(int m, long long n_rb, long long n_kb) {\n'
                   "  const Plan p = plan(m, n_rb, n_kb);\n  return p.tok * 16 + p.C;\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-fsanitize=signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.x_of.restype = ctypes.c_longlong
    lib.x_of.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    lib.plan_of.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_longlong]
    return lib


def _kbs():
    """Channel blocks up to 2^28 channels, and every place where a size in 32 bits would change its sign or be zero."""
    out = set(range(1, 300))
    for e in range(8, 22):
        out |= {(1 << e) + d for d in (-9, -8, -4, -1, 0, 1, 3, 4, 8)}
    return sorted(k for k in out if k <= 1 << 21)


def test_bytes_of_x(L):
    for n_kb in _kbs():
        for C in (4, 8):
            for tok in (16, 32):
                share = -(-n_kb // C) * tok * 128 * 2
                assert L.x_of(n_kb, C, tok) == -(-share // 1024) * 1024


def test_no_plan_passes_what_a_cluster_holds(L):
    taken = set()
    for n_kb in _kbs():
        for n_rb in (1, 2, 7, 64, 1000, 31250, 1 << 23):
            for m in range(1, 33):
                v = L.plan_of(m, n_rb, n_kb)
                tok, C = v // 16, v % 16
                blocks = n_rb * n_kb
                worth = (m > 24 and blocks >= 2048 and n_kb >= 16) or (m > 16 and blocks >= 2048 and n_kb >= 32) \
                    or (m > 8 and blocks >= 16384 and n_kb >= 64)
                fits = [(t, c) for t in ((32, 16) if m > 16 else (16,)) for c in (4, 8)
                        if -(-n_kb // c) * t * 256 <= X_BYTES]
                assert (tok, C) == (fits[0] if worth and fits else (0, 0)), (m, n_rb, n_kb)
                taken.add((tok, C))
                if tok:                                       # each CTA of a cluster has two channel blocks and more
                    assert n_kb >= 2 * C
    assert taken == {(0, 0), (16, 4), (16, 8), (32, 4), (32, 8)}


def test_the_largest_channels_go_to_the_form_without_clusters_of_x(L):
    for m in (17, 32):
        for n_kb in (1 << 20, (1 << 20) + 1, 1 << 21):       # n_in = 2^27 .. 2^28
            assert L.plan_of(m, 1, n_kb) == 0
