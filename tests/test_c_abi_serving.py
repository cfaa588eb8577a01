"""The structures of the norm/rotation and paged-cache calls: a C program and the ctypes binding agree on sizes and
offsets, and a plain C caller reaches the host-only calls and the argument checks."""
import ctypes
import os
import shutil
import subprocess

import pytest

import long_context_prefill_moba_b200 as M
from long_context_prefill_moba_b200 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.join(ROOT, "long_context_prefill_moba_b200")

PROGRAM = r"""
#include <stddef.h>
#include <stdio.h>
#include "moba.h"
#define AT(t, f) printf(#t "." #f " %zu\n", offsetof(t, f))
int main(void) {
  moba_rope_shape_t r = {8, 32, 8, 128, MOBA_BF16, 0, 0, {128, 0, MOBA_F32, 1e-6f}};
  moba_paged_shape_t p = {4, 8, 32, 8, 128, 64, 100, 16, MOBA_BF16, 0.0f, 0, 0, 0, 0, 0};
  if (moba_check_rope_shape(&r) != MOBA_OK || moba_check_paged_shape(&p) != MOBA_OK) return 1;
  if (moba_qk_norm_rope_bwd_workspace_size(&r) == 0 || moba_paged_attn_workspace_size(&p) == 0) return 2;
  if (moba_qk_norm_rope(&r, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL) != MOBA_ERR_INVALID_ARG) return 3;
  if (moba_paged_append(&p, &r.rope, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL) !=
      MOBA_ERR_INVALID_ARG)
    return 4;
  if (moba_paged_attn(&p, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0, NULL) != MOBA_ERR_INVALID_ARG) return 5;
  printf("sizes %zu %zu %zu\n", sizeof(moba_rope_t), sizeof(moba_rope_shape_t), sizeof(moba_paged_shape_t));
  AT(moba_rope_t, eps); AT(moba_rope_shape_t, dtype); AT(moba_rope_shape_t, q_stride); AT(moba_rope_shape_t, rope);
  AT(moba_paged_shape_t, page_size); AT(moba_paged_shape_t, scale); AT(moba_paged_shape_t, q_stride);
  AT(moba_paged_shape_t, v_page_stride);
  return 0;
}
"""


@pytest.mark.parametrize("compiler,flags", [("gcc", ["-std=c99", "-pedantic"]), ("g++", ["-std=c++17"])])
def test_structures_agree(tmp_path, compiler, flags):
    if shutil.which(compiler) is None:
        pytest.skip(f"{compiler} not available")
    B.build()
    src = tmp_path / ("prog.c" if compiler == "gcc" else "prog.cpp")
    src.write_text(PROGRAM)
    exe = tmp_path / "prog"
    subprocess.run([compiler, *flags, "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-L", LIBDIR,
                    "-lmoba", f"-Wl,-rpath,{LIBDIR}", "-o", str(exe)], check=True, capture_output=True, text=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, (res.returncode, res.stdout, res.stderr)
    lines = res.stdout.split("\n")
    assert lines[0] == "sizes %d %d %d" % tuple(ctypes.sizeof(t) for t in (M.MobaRope, M.MobaRopeShape, M.MobaPagedShape))
    types = {"moba_rope_t": M.MobaRope, "moba_rope_shape_t": M.MobaRopeShape, "moba_paged_shape_t": M.MobaPagedShape}
    for line in lines[1:-1]:
        name, at = line.split()
        t, field = name.split(".")
        assert getattr(types[t], field).offset == int(at), line
