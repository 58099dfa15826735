"""Host-side checks of the sorted-row and adapter entry points that need no GPU: null
handles, refused descriptions, struct layouts."""
import ctypes
import os
import shutil
import subprocess

import pytest

import w4a16_quantized_expert_b200 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def create(**kw):
    d = dict(in_features=64, out_features=32, n_adapters=4, max_rank=16, dtype=0, max_tokens=8)
    w = dict(a=0x1000, b=0x2000, scaling=0x3000, rank=None)
    for k, v in kw.items():
        (d if k in d else w)[k] = v
    desc, wt, h = moe.moe_adapters_desc(**d), moe.moe_adapters_weights(**w), ctypes.c_void_p(1)
    rc = moe.lib().moe_adapters_create(ctypes.byref(desc), ctypes.byref(wt), ctypes.byref(h))
    return rc, h.value


@pytest.mark.parametrize("bad", [
    dict(in_features=0), dict(in_features=60), dict(in_features=16392), dict(out_features=0), dict(out_features=16385),
    dict(n_adapters=0), dict(n_adapters=1025), dict(max_rank=0), dict(max_rank=12), dict(max_rank=136), dict(dtype=2),
    dict(dtype=-1), dict(max_tokens=0), dict(max_tokens=65537), dict(a=None), dict(a=0x1008), dict(b=None),
    dict(b=0x2002), dict(scaling=None), dict(scaling=0x3004), dict(rank=0x4004),
])
def test_create_refuses(bad):
    assert create(**bad) == (moe.MOE_ERR_INVALID_ARG, None)


def test_null_handles():
    L, none = moe.lib(), None
    bad = moe.MOE_ERR_INVALID_ARG
    assert L.moe_sorted_rows(none, 1, 1) == 0 and L.moe_sort_workspace_size(none, 1) == 0
    assert L.moe_sort_tokens(none, none, 0, 0, none, 1, 1, none, 0, none, none, none, none, 0, none) == bad
    assert L.moe_sort_tokens_backward(none, none, 0, 0, none, 1, none, 0, 0, none) == bad
    assert L.moe_unsort_tokens(none, none, 0, 0, none, none, none, 1, none, 0, 0, none) == bad
    assert L.moe_unsort_tokens_backward(none, none, 0, 0, none, 0, 0, none, none, none, none, 1, none, none,
                                        none) == bad
    assert L.moe_adapters_workspace_size(none, 1) == 0
    assert L.moe_adapters_apply(none, none, 0, none, 1, none, 0, none, 0, 0, none, none, 0, none) == bad
    assert L.moe_adapters_backward(none, none, 0, none, none, 0, none, 1, none, 0, none, 0, 0, none, none, 0, none, 0,
                                   none) == bad
    assert L.moe_adapters_destroy(none) == moe.MOE_OK
    st = ctypes.c_int(0)
    assert L.moe_adapters_get_device_status(none, ctypes.byref(st)) == bad
    assert L.moe_adapters_create(none, none, none) == bad


def test_struct_layouts_match_the_header(tmp_path):
    if not shutil.which("gcc"):
        pytest.skip("no host C compiler")
    structs = ("moe_adapters_desc", "moe_adapters_weights")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe.h"', "int main(void) {"]
    want = []
    for s in structs:
        c = getattr(moe, s)
        lines.append(f'  printf("%zu\\n", sizeof({s}));')
        want.append(ctypes.sizeof(c))
        for f, _ in c._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({s}, {f}));')
            want.append(getattr(c, f).offset)
    lines += ['  printf("%d %d %d\\n", MOE_DTYPE_F16, MOE_DTYPE_BF16, MOE_DTYPE_F32);', "  return 0;", "}"]
    want += [moe.MOE_DTYPE_F16, moe.MOE_DTYPE_BF16, moe.MOE_DTYPE_F32]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines) + "\n")
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    assert [int(v) for v in subprocess.check_output([str(exe)], text=True).split()] == want
