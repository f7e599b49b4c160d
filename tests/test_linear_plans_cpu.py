"""Which kernel a linear layer's shape takes (error_compensated_bit_02_amd/csrc/layer_plan.h,
plain C++), so that the GPU tests' shapes reach every one."""
import ctypes
import os
import shutil
import subprocess

import pytest

import linear_cases as cases
from error_compensated_bit_02_amd import binding

F32, BF16 = cases.F32, cases.BF16
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "error_compensated_bit_02_amd", "csrc")
DRIVER = r"""
#include <cstdio>
#include "layer_plan.h"
int main() {
  long long rows, out, in;
  int f32, weight_f32, aligned, back;
  while (std::scanf("%lld %lld %lld %d %d %d %d", &rows, &out, &in, &f32, &weight_f32, &aligned, &back) == 7) {
    const ob::LayerPlan p = ob::layer_plan({rows, out, in, f32 != 0, weight_f32 != 0, aligned != 0, back != 0});
    std::printf("%d %d %d %d %lld\n", p.tile, p.splits, p.pack_a, p.pack_b,
                static_cast<long long>(p.a_bytes + p.b_bytes + p.part_bytes));
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("layer_plan")
    src, exe = d / "driver.cpp", d / "driver"
    src.write_text(DRIVER)
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def ask(shapes):
        """[(tile, slices, A copied, B copied, bytes)] of (xt, lt, back, rows, out, in) with contiguous rows."""
        text = ""
        for xt, lt, back, rows, out, inp in shapes:
            aligned = (out if back else inp) * (4 if xt == F32 else 2) % 16 == 0 or rows <= 1
            text += f"{rows} {out} {inp} {int(xt == F32)} {int(lt == F32)} {int(aligned)} {int(back)}\n"
        got = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
        return [tuple(map(int, line.split())) for line in got if line]
    return ask


def test_the_shapes_reach_every_kernel(plans):
    """Both directions of four pairs of types: three tiles each, in one slice and in several."""
    for (xt, lt, back), by in cases.PLANS.items():
        got = plans([(xt, lt, back, *s) for s in by.values()])
        for (tile, sliced, pa, pb), shape, (t, splits, a, b, _) in zip(by, by.values(), got):
            assert (t, splits > 1, a, b) == (tile, sliced, pa, pb), (xt, lt, back, shape, t, splits, a, b)
        assert {k[:2] for k in by} == {(t, s) for t in (0, 1, 2) for s in (False, True)}
    assert len(cases.PLANS) == 8
    for xt, lt, back in cases.PLANS:
        got = plans([(xt, lt, back, *s) for s in cases.FEW[back]])
        assert all(t == -1 for t, *_ in got) and {s > 1 for _, s, *_ in got} == ({False, True} if back else {False})


def test_the_header_is_what_the_library_asks(plans):
    lib, n = binding.load_library(), ctypes.c_int64()
    shapes = cases.shapes()
    for (xt, lt, back, rows, out, inp), got in zip(shapes, plans(shapes)):
        code = {F32: 0, BF16: 1}
        aligned = (out if back else inp) * (4 if xt == F32 else 2) % 16 == 0 or rows <= 1
        assert lib.ob_linear_work(rows, out, inp, code[xt], code[lt], int(aligned), int(back), ctypes.byref(n)) == 0
        assert n.value == got[-1]
