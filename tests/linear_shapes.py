"""Which kernel a linear layer's call takes: the library's own rule (csrc/linear_shape.h,
plain C++), compiled by itself."""
import ctypes
import os
import subprocess
import tempfile

from conftest import ROOT

TILES = ["256x256", "128x128", "64x64 pair", "64x64 quad", "288x256"]
SOURCE = """
#include "linear_shape.h"
extern "C" {
int forward(int rows, int E, int grouped, int N, int K, int gated, int cus) {
  const moe::LinearSizes a = {rows, E, grouped != 0, N, K, gated != 0};
  const moe::StreamItem few = moe::stream_item(a, cus);
  return few.nb ? 100 + 10 * few.nb + few.mb : (int)moe::forward_tile(a, cus);
}
int grad_x(int rows, int E, int grouped, int N, int K, int gated, int cus) {
  return moe::grad_x_tile({rows, E, grouped != 0, N, K, gated != 0}, cus);
}
int grad_w(int rows, int E, int grouped, int N, int K, int gated, int cus) {
  return moe::grad_w_tile({rows, E, grouped != 0, N, K, gated != 0}, cus);
}
}
"""
_lib = None


def picked(op, rows, E, N, K, act="none", cus=256):
    """The tile that `op` (forward, grad_x, grad_w) of these sizes takes, a name of TILES, or
    "stream NB.MB"; E = 0: plain rows."""
    global _lib
    if _lib is None:
        with tempfile.TemporaryDirectory() as d:
            src, so = os.path.join(d, "rule.cpp"), os.path.join(d, "rule.so")
            with open(src, "w") as f:
                f.write(SOURCE)
            subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-I",
                            os.path.join(ROOT, "mixture_experts_layer_lds_amd", "csrc"), src, "-o", so], check=True)
            _lib = ctypes.CDLL(so)
    got = getattr(_lib, op)(rows, max(1, E), int(E > 0), N, K, int(act == "swiglu"), cus)
    return TILES[got] if got < 100 else f"stream {(got - 100) // 10}.{got % 10}"
