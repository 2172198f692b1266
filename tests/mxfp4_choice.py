"""Which kernel a call of the MXFP4 products takes: the library's own choice (csrc/mxfp4_shapes.h), compiled for the host."""
import ctypes
import os
import subprocess

import pytest

from token_dispatch_expert_amd import build

CUS = 256  # of an MI355X

SOURCE = r"""
#include "mxfp4_shapes.h"
using namespace moe;
template <bool X4>
static int gemm(const MxGemmArgs& a) { return a.g.b2 ? pick_gemm<X4, true>(a, %(cus)d) : pick_gemm<X4, false>(a, %(cus)d); }
template <typename T>
constexpr int length(const T& t) { return sizeof(t) / sizeof(Shape); }
extern "C" {
int gemm_shape(int x4, int pair, int codes, int rows, int E, int N, int K) {
  MxGemmArgs a{};
  a.g.rows = rows, a.g.E = E, a.g.N = N, a.g.K = K;
  a.g.b2 = pair ? &a : nullptr;
  a.out_scales = codes ? reinterpret_cast<uint8_t*>(&a) : nullptr;
  return x4 ? gemm<true>(a) : gemm<false>(a);
}
int dgrad_shape(int pair, int rows, int E, int N, int K) {
  GroupedGemmArgs g{};
  g.rows = rows, g.E = E, g.N = N, g.K = K;
  g.b2 = pair ? &g : nullptr;
  return pick_dgrad(g, %(cus)d);
}
int gemm_shapes(int x4, int pair) {
  return x4 ? (pair ? length(GemmShapes<true, true>::all) : length(GemmShapes<true, false>::all))
            : (pair ? length(GemmShapes<false, true>::all) : length(GemmShapes<false, false>::all));
}
int holds_groups(int x4, int i) { return x4 ? GemmShapes<true, true>::all[i].groups : GemmShapes<false, true>::all[i].groups; }
int dgrad_shapes() { return kDgradShapeCount; }
}
"""


def load(folder):
    """The choice as a library: gemm_shape(4-bit rows, gate and up, h in codes, rows, E, N, K), dgrad_shape(two, rows, E, N, K),
    how many shapes there are, and whether one holds the groups of h in codes."""
    if not os.path.exists(build._hipcc()):
        pytest.skip(f"needs {build._hipcc()}")
    src, lib = os.path.join(folder, "choice.hip"), os.path.join(folder, "choice.so")
    with open(src, "w") as f:
        f.write(SOURCE % dict(cus=CUS))
    flags = [f for f in build.FLAGS if f != "-O3"]
    r = subprocess.run([build._hipcc(), *flags, "-O1", "--offload-host-only", "-shared", "-x", "hip", src, "-o", lib], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(lib)
