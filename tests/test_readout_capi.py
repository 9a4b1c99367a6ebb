"""The readout's C entry points check every argument before anything is launched (no GPU needed), and their
config structs have the C layout."""
import ctypes
import os
import subprocess

import pytest

from hierarchical_kv_routing_tok_b200 import _capi as C
from hierarchical_kv_routing_tok_b200 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ODD = 1 << 20, (1 << 20) + 8                       # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return C.load()


def packed(**kw):
    base = dict(Hq=32, Hkv=8, D=128, n_seqs=3, total=1000, dtype=C.HGA_BF16)
    base.update(kw)
    return C.PackedConfig(**base)


def pages(**kw):
    base = dict(n_layers=2, n_pages=100, page=64, Hkv=8, D=128, max_seqs=4, max_pages=10, dtype=C.HGA_BF16)
    base.update(kw)
    return C.PagesConfig(**base)


@pytest.mark.parametrize("cls,name", [(C.PackedConfig, "hga_packed_config_t"), (C.PagesConfig, "hga_pages_config_t")])
def test_struct_layout_matches_c(tmp_path, cls, name):
    src = tmp_path / "layout.c"
    fields = [n for n, _ in cls._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "hga.h"\nint main(void){\n'
                   f'  printf("%zu\\n", sizeof({name}));\n'
                   + "".join(f'  printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    vals = [int(v) for v in subprocess.check_output([str(exe)], text=True).split()]
    assert vals == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


def code(call):
    with pytest.raises(C.HGAError) as e:
        call()
    return e.value.code


@pytest.mark.parametrize("kw,want", [
    (dict(Hq=30), C.HGA_ERR_ARG), (dict(Hkv=0), C.HGA_ERR_ARG), (dict(Hq=0), C.HGA_ERR_ARG),
    (dict(D=64), C.HGA_ERR_UNSUPPORTED), (dict(n_seqs=-1), C.HGA_ERR_ARG), (dict(total=-1), C.HGA_ERR_ARG),
    (dict(total=2 ** 31 - 1), C.HGA_ERR_UNSUPPORTED), (dict(n_seqs=2 ** 25), C.HGA_ERR_UNSUPPORTED),
    (dict(dtype=5), C.HGA_ERR_ARG), (dict(flags=8), C.HGA_ERR_ARG), (dict(reserved=1), C.HGA_ERR_ARG),
    (dict(q_stride_t=64), C.HGA_ERR_ARG), (dict(k_stride_h=-128), C.HGA_ERR_ARG), (dict(v_stride_t=1 << 50), C.HGA_ERR_ARG),
    (dict(k_stride_t=1028), C.HGA_ERR_ALIGN), (dict(softmax_scale=-1.0), C.HGA_ERR_ARG),
    (dict(softmax_scale=float("nan")), C.HGA_ERR_ARG), (dict(softmax_scale=float("inf")), C.HGA_ERR_ARG),
    (dict(wait_limit_ns=-1), C.HGA_ERR_ARG),
])
def test_packed_config(kw, want):
    assert code(lambda: C.packed_workspace_size(packed(**kw))) == want
    c = packed(**kw)
    assert code(lambda: C.packed_attn_fwd(c, *[OK] * 8)) == want
    assert code(lambda: C.packed_attn_bwd(c, *[OK] * 12)) == want


def test_packed_pointers():
    c = packed()
    for call, n in ((C.packed_attn_fwd, 7), (C.packed_attn_bwd, 11)):
        for i in range(n):
            args = [OK] * n
            args[i] = None
            if i != 5:                                 # o_lo may be left out
                assert code(lambda: call(c, *args, OK)) == C.HGA_ERR_ARG
            args[i] = ODD if i != 3 else OK + 2
            assert code(lambda: call(c, *args, OK)) == C.HGA_ERR_ALIGN
        assert code(lambda: call(c, *[OK] * n, None)) == C.HGA_ERR_WORKSPACE
        assert code(lambda: call(c, *[OK] * n, ODD)) == C.HGA_ERR_ALIGN


def test_packed_workspace_grows():
    a, b = C.packed_workspace_size(packed()), C.packed_workspace_size(packed(total=100000, n_seqs=1000))
    assert a % 256 == 0 and b > a >= 256 + 32 * 1000 * 4
    assert C.packed_workspace_size(packed(total=0, n_seqs=0)) >= 256


@pytest.mark.parametrize("kw,want", [
    (dict(n_layers=0), C.HGA_ERR_ARG), (dict(n_pages=0), C.HGA_ERR_ARG), (dict(page=24), C.HGA_ERR_UNSUPPORTED),
    (dict(page=256), C.HGA_ERR_UNSUPPORTED), (dict(D=64), C.HGA_ERR_UNSUPPORTED), (dict(max_seqs=9000), C.HGA_ERR_UNSUPPORTED),
    (dict(n_pages=2 ** 21), C.HGA_ERR_UNSUPPORTED), (dict(max_pages=2 ** 26), C.HGA_ERR_UNSUPPORTED),
    (dict(dtype=9), C.HGA_ERR_ARG), (dict(page_stride=100), C.HGA_ERR_ARG), (dict(page_stride=65536 + 4), C.HGA_ERR_ALIGN),
    (dict(layer_stride=65536), C.HGA_ERR_ARG),           # layers that overlap
    (dict(layer_stride=-65536), C.HGA_ERR_ARG), (dict(wait_limit_ns=-5), C.HGA_ERR_ARG),
])
def test_pages_config(kw, want):
    c = pages(**kw)
    assert code(lambda: C.pages_workspace_size(c)) == want
    assert code(lambda: C.pages_reserve(c, 1, *[OK] * 7)) == want
    assert code(lambda: C.pages_free(c, 1, *[OK] * 5)) == want
    assert code(lambda: C.pages_compact(c, *[OK] * 7)) == want
    assert code(lambda: C.paged_attn(c, 0, 1, 32, 0.0, OK, OK, 0, *[OK] * 7)) == want


def test_pages_calls():
    c = pages()
    assert C.pages_workspace_size(c) > 0
    attn = lambda layer=0, n=1, Hq=32, scale=0.0, stride=0, ptrs=(OK,) * 9: C.paged_attn(
        c, layer, n, Hq, scale, ptrs[0], ptrs[1], stride, *ptrs[2:])
    for kw, want in ((dict(layer=2), C.HGA_ERR_ARG), (dict(layer=-1), C.HGA_ERR_ARG), (dict(n=-1), C.HGA_ERR_ARG),
                     (dict(n=8193), C.HGA_ERR_UNSUPPORTED), (dict(Hq=12), C.HGA_ERR_ARG), (dict(Hq=0), C.HGA_ERR_ARG),
                     (dict(Hq=8 * 129), C.HGA_ERR_UNSUPPORTED), (dict(scale=float("nan")), C.HGA_ERR_ARG),
                     (dict(stride=128), C.HGA_ERR_ARG), (dict(stride=4100), C.HGA_ERR_ALIGN)):
        assert code(lambda: attn(**kw)) == want, kw
    for i in range(8):
        ptrs = [OK] * 9
        ptrs[i] = None
        assert code(lambda: attn(ptrs=ptrs)) == C.HGA_ERR_ARG, i
        ptrs[i] = OK + 2
        assert code(lambda: attn(ptrs=ptrs)) == C.HGA_ERR_ALIGN, i
    assert code(lambda: attn(ptrs=[OK] * 8 + [None])) == C.HGA_ERR_WORKSPACE
    assert code(lambda: C.pages_write(c, 5, 1, OK, OK, OK, 3, OK, 0, 0, OK, 0, 0, *[OK] * 5)) == C.HGA_ERR_ARG
    assert code(lambda: C.pages_write(c, 0, 1, OK, OK, OK, 3, OK, 1020, 0, OK, 0, 0, *[OK] * 5)) == C.HGA_ERR_ALIGN
    assert code(lambda: C.pages_write(c, 0, 1, OK, OK, OK, -3, OK, 0, 0, OK, 0, 0, *[OK] * 5)) == C.HGA_ERR_ARG
    assert code(lambda: C.pages_write(c, 0, 1, OK, None, OK, 3, OK, 0, 0, OK, 0, 0, *[OK] * 5)) == C.HGA_ERR_ARG
    assert code(lambda: C.pages_fork(c, 1, OK, OK, OK, OK, None, OK, OK, OK)) == C.HGA_ERR_ARG
    assert code(lambda: C.pages_fork(c, 1, OK, OK, OK, OK, OK, OK, OK, None)) == C.HGA_ERR_WORKSPACE
    assert code(lambda: C.pages_copy(c, 1, OK, OK, ODD, OK, OK)) == C.HGA_ERR_ALIGN
    assert code(lambda: C.pages_copy(c, -1, OK, OK, OK, OK, OK)) == C.HGA_ERR_ARG
    # nothing to do: nothing is launched
    C.pages_reserve(c, 0, None, None, None, OK, OK, OK, OK)
    C.pages_free(c, 0, None, OK, OK, OK, OK)
    C.pages_copy(c, 0, None, None, OK, OK, OK)
    attn(n=0, ptrs=(None, None, OK, OK, OK, OK, None, None, OK))


def test_layers_side_by_side_are_accepted():
    data = 8 * 64 * 128
    assert C.pages_workspace_size(pages(page_stride=4 * data, layer_stride=2 * data)) > 0
    assert C.pages_workspace_size(pages(page_stride=4 * data, layer_stride=400 * data)) > 0
    assert code(lambda: C.pages_workspace_size(pages(page_stride=2 * data, layer_stride=2 * data))) == C.HGA_ERR_ARG
