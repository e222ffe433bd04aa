"""Refusals of the grouped products: before any launch, so without a GPU."""

import ctypes as C
import os

import pytest
import torch

from newton_schulz_10_b200 import build as nbuild
from newton_schulz_10_b200 import muon as mu

FAKE = 1 << 20  # 16-byte aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mu.LIB_PATH):
        nbuild.build()
    return mu.lib()


def desc(**kw):
    g = dict(dtype=mu.BF16, experts=2, tokens=10, n=16, k=24, ldx=24, ldy=16, ldw=24, w_stride=16 * 24, offsets=FAKE, dev_status=None)
    g.update(kw)
    return mu.Grouped(**g)


BAD = [
    (dict(dtype=mu.F32), mu.ERR_DTYPE),
    (dict(dtype=9), mu.ERR_DTYPE),
    (dict(experts=-1), mu.ERR_SHAPE),
    (dict(experts=1025), mu.ERR_SHAPE),
    (dict(tokens=-1), mu.ERR_SHAPE),
    (dict(tokens=2 ** 31), mu.ERR_SHAPE),
    (dict(n=0), mu.ERR_SHAPE),
    (dict(k=0), mu.ERR_SHAPE),
    (dict(ldx=16), mu.ERR_SHAPE),
    (dict(ldy=8), mu.ERR_SHAPE),
    (dict(ldw=16), mu.ERR_SHAPE),
    (dict(w_stride=0), mu.ERR_SHAPE),
    (dict(w_stride=15 * 24), mu.ERR_SHAPE),
    (dict(k=23, ldx=23), mu.ERR_ALIGN),
    (dict(n=15, ldy=15), mu.ERR_ALIGN),
    (dict(k=20, ldw=20), mu.ERR_ALIGN),
    (dict(w_stride=16 * 24 + 4), mu.ERR_ALIGN),
    (dict(offsets=None), mu.ERR_INVALID_ARG),
    (dict(offsets=FAKE + 2), mu.ERR_ALIGN),
    (dict(dev_status=FAKE + 2), mu.ERR_ALIGN),
    (dict(tokens=2 ** 31 - 1, n=2 ** 20, ldy=2 ** 20, w_stride=2 ** 20 * 24), mu.ERR_SHAPE),
]


@pytest.mark.parametrize("kw,want", BAD, ids=[str(b[0]) for b in BAD])
def test_refused(L, kw, want):
    g = desc(**kw)
    assert L.grouped_matmul(C.byref(g), FAKE, FAKE, FAKE, None) == want
    assert L.grouped_matmul_dx(C.byref(g), FAKE, FAKE, FAKE, None) == want
    assert L.grouped_matmul_dw(C.byref(g), FAKE, FAKE, FAKE, mu.BF16, 1.0, 0.0, FAKE, 1 << 20, None) == want


def test_refused_pointers(L):
    g = desc()
    for call in (L.grouped_matmul, L.grouped_matmul_dx):
        for i in range(3):
            args = [FAKE] * 3
            args[i] = None
            assert call(C.byref(g), *args, None) == mu.ERR_INVALID_ARG
            args[i] = FAKE + 8
            assert call(C.byref(g), *args, None) == mu.ERR_ALIGN
        assert call(None, FAKE, FAKE, FAKE, None) == mu.ERR_INVALID_ARG
    dw = lambda g, a, b, c, t, alpha, beta, ws, nb: L.grouped_matmul_dw(C.byref(g), a, b, c, t, alpha, beta, ws, nb, None)
    need = mu.grouped_workspace_size(2)
    assert dw(g, FAKE, FAKE, FAKE, mu.F32, 1.0, 0.0, None, need) == mu.ERR_WORKSPACE
    assert dw(g, FAKE, FAKE, FAKE, mu.F32, 1.0, 0.0, FAKE, need - 1) == mu.ERR_WORKSPACE
    assert dw(g, FAKE, FAKE, FAKE, mu.F16, 1.0, 0.0, FAKE, need) == mu.ERR_DTYPE
    assert dw(g, FAKE, FAKE, FAKE, 7, 1.0, 0.0, FAKE, need) == mu.ERR_DTYPE
    assert dw(g, FAKE, FAKE, FAKE, mu.F32, float("nan"), 0.0, FAKE, need) == mu.ERR_INVALID_ARG
    assert dw(g, FAKE, FAKE, FAKE, mu.F32, 1.0, float("inf"), FAKE, need) == mu.ERR_INVALID_ARG
    assert dw(g, None, FAKE, FAKE, mu.F32, 1.0, 0.0, FAKE, need) == mu.ERR_INVALID_ARG
    assert dw(g, FAKE, FAKE, FAKE + 4, mu.F32, 1.0, 0.0, FAKE, need) == mu.ERR_ALIGN
    assert mu.grouped_workspace_size(-1) == 0 and mu.grouped_workspace_size(1025) == 0


def test_nothing_to_do(L):
    for kw in (dict(experts=0), dict(tokens=0)):
        g = desc(**kw)
        assert L.grouped_matmul(C.byref(g), None, None, None, None) == mu.OK
        assert L.grouped_matmul_dx(C.byref(g), None, None, None, None) == mu.OK
    assert L.grouped_matmul_dw(C.byref(desc(experts=0)), None, None, None, mu.F32, 1.0, 0.0, None, 0, None) == mu.OK


def test_struct_layout_matches_c(tmp_path):
    import subprocess
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "muon.h"\nint main(void){printf("%zu %zu %zu\\n",'
                   "sizeof(muon_grouped), offsetof(muon_grouped, ldw), offsetof(muon_grouped, dev_status));return 0;}\n")
    subprocess.run(["gcc", "-I", inc, str(src), "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    assert list(map(int, got)) == [C.sizeof(mu.Grouped), mu.Grouped.ldw.offset, mu.Grouped.dev_status.offset]


def test_binding_refuses_wrong_tensors(L):
    x, w, off = torch.zeros(10, 24, dtype=torch.bfloat16), torch.zeros(2, 16, 24, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    cases = [
        (lambda: mu.grouped_matmul(x, w, off), mu.ERR_INVALID_ARG),  # not on a GPU
        (lambda: mu.grouped_matmul(x[:, :16], w, off), mu.ERR_SHAPE),
        (lambda: mu.grouped_matmul(x[0], w, off), mu.ERR_SHAPE),
        (lambda: mu.grouped_matmul(x, w, off[:2]), mu.ERR_SHAPE),
        (lambda: mu.grouped_matmul(x, w.half(), off), mu.ERR_DTYPE),
        (lambda: mu.grouped_matmul(x.float(), w.float(), off), mu.ERR_DTYPE),
        (lambda: mu.grouped_matmul(x, w, off.long()), mu.ERR_DTYPE),
        (lambda: mu.grouped_matmul_dx(x, w, off), mu.ERR_SHAPE),
        (lambda: mu.grouped_matmul_dw(x, x, off, beta=0.5), mu.ERR_INVALID_ARG),
    ]
    for i, (call, code) in enumerate(cases):
        with pytest.raises(mu.MuonError) as err:
            call()
        assert err.value.code == code, i


@pytest.mark.parametrize("tokens", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 255, 2 ** 31 - 512])
def test_rows_whose_tiles_leave_32_bits_are_refused(L, tokens):
    """Row numbers rounded up to a tile, or to a block of 64, have to stay within 32 bits."""
    g = desc(tokens=tokens, n=8, k=8, ldx=8, ldy=8, ldw=8, w_stride=64)
    for call in (L.grouped_matmul, L.grouped_matmul_dx):
        assert call(C.byref(g), FAKE, FAKE, FAKE, None) == mu.ERR_SHAPE
    assert L.grouped_matmul_dw(C.byref(g), FAKE, FAKE, FAKE, mu.F32, 1.0, 0.0, FAKE, 1 << 30, None) == mu.ERR_SHAPE
