"""Refusals of the stack update: before any launch, so without a GPU."""

import ctypes as C
import os
import subprocess

import pytest
import torch

from newton_schulz_10_b200 import build as nbuild
from newton_schulz_10_b200 import muon as mu

FAKE = 1 << 20  # never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mu.LIB_PATH):
        nbuild.build()
    return mu.lib()


def stack(**kw):
    s = dict(W=FAKE, M=FAKE, G=FAKE, copy=None, w_dtype=mu.F32, g_dtype=mu.BF16, copy_dtype=0, count=3, rows=32, cols=48,
             w_stride=32 * 48, w_ld=48, m_stride=32 * 48, m_ld=48, g_stride=32 * 48, g_ld=48, copy_stride=32 * 48, copy_ld=48)
    s.update(kw)
    return (mu.StackArray * 1)(mu.StackArray(**s))


def call(L, s, p, ws=FAKE, nbytes=1 << 30, count=1):
    return L.muon_stack_step(s, count, C.byref(p), ws, nbytes, None)


BAD = [
    (dict(W=None), mu.ERR_INVALID_ARG),
    (dict(M=None), mu.ERR_INVALID_ARG),
    (dict(w_dtype=mu.F16X2), mu.ERR_DTYPE),
    (dict(g_dtype=9), mu.ERR_DTYPE),
    (dict(copy=FAKE, copy_dtype=mu.F32), mu.ERR_DTYPE),
    (dict(W=FAKE + 2), mu.ERR_ALIGN),
    (dict(M=FAKE + 2), mu.ERR_ALIGN),
    (dict(G=FAKE + 1), mu.ERR_ALIGN),
    (dict(copy=FAKE + 1, copy_dtype=mu.BF16), mu.ERR_ALIGN),
    (dict(count=-1), mu.ERR_SHAPE),
    (dict(rows=-1), mu.ERR_SHAPE),
    (dict(cols=-1), mu.ERR_SHAPE),
    (dict(count=65536), mu.ERR_SHAPE),
    (dict(w_ld=47), mu.ERR_SHAPE),
    (dict(m_ld=40), mu.ERR_SHAPE),
    (dict(w_stride=0), mu.ERR_SHAPE),
    (dict(w_stride=32 * 48 - 1), mu.ERR_SHAPE),  # overlapping matrices
    (dict(w_stride=47, w_ld=400), mu.ERR_SHAPE),  # overlapping column blocks
    (dict(w_stride=48, w_ld=143), mu.ERR_SHAPE),
    (dict(m_stride=0), mu.ERR_SHAPE),
    (dict(g_stride=-1), mu.ERR_SHAPE),
    (dict(copy=FAKE, copy_dtype=mu.BF16, copy_stride=0), mu.ERR_SHAPE),
    (dict(rows=2 ** 31 - 1, count=2), mu.ERR_SHAPE),
]


@pytest.mark.parametrize("kw,want", BAD, ids=[str(b[0]) for b in BAD])
def test_refused(L, kw, want):
    assert call(L, stack(**kw), mu.stack_params()) == want


def test_accepted_layouts_reach_the_workspace_check(L):
    p = mu.stack_params()
    for kw in (dict(), dict(w_stride=48, w_ld=144), dict(g_stride=0), dict(g_ld=0), dict(count=1, w_stride=0, m_stride=-5),
               dict(rows=1, w_ld=0, m_ld=0, w_stride=48, m_stride=48), dict(W=FAKE + 4, M=FAKE + 4, G=FAKE + 2)):
        assert call(L, stack(**kw), p, None, 0) == mu.ERR_WORKSPACE, kw
        assert call(L, stack(**kw), p, FAKE, 1024) == mu.ERR_WORKSPACE
        assert call(L, stack(**kw), p, FAKE + 8) == mu.ERR_ALIGN


def test_refused_parameters(L):
    s = stack()

    def bad(**kw):
        p = mu.stack_params()
        for name, v in kw.items():
            setattr(p, name, v)
        return call(L, s, p)

    nan = float("nan")
    for name in ("mu", "lr", "weight_decay", "scale"):
        assert bad(**{name: nan}) == mu.ERR_INVALID_ARG
    assert bad(nesterov=2) == mu.ERR_INVALID_ARG
    assert bad(dev_status=FAKE + 2) == mu.ERR_ALIGN
    assert call(L, stack(G=None), mu.stack_params(nesterov=True)) == mu.ERR_INVALID_ARG
    assert call(L, s, mu.stack_params(ns=mu.ns_params(compute=mu.F16X2, gram=True))) == mu.ERR_UNSUPPORTED
    assert call(L, s, mu.stack_params(ns=mu.ns_params(compute=7))) == mu.ERR_DTYPE
    assert call(L, s, mu.stack_params(ns=mu.ns_params(T=0))) == mu.ERR_INVALID_ARG
    assert call(L, s, mu.stack_params(), count=-1) == mu.ERR_INVALID_ARG
    assert L.muon_stack_step(None, 1, C.byref(mu.stack_params()), FAKE, 1 << 30, None) == mu.ERR_INVALID_ARG
    assert L.muon_stack_workspace_size(s, 1, C.byref(mu.stack_params(ns=mu.ns_params(T=17)))) == 0


def test_nothing_to_do(L):
    p = mu.stack_params()
    assert call(L, stack(), p, None, 0, count=0) == mu.OK
    for kw in (dict(count=0), dict(rows=0), dict(cols=0)):
        assert call(L, stack(W=None, M=None, **kw), p, None, 0) == mu.OK


def test_two_planes_stay_out_of_the_other_entry_points(L):
    ns = mu.ns_params(compute=mu.F16X2)
    assert mu.ns_workspace_size(64, 64, ns) == 0
    assert L.ns_polar(FAKE, mu.F32, FAKE, mu.F32, 64, 64, C.byref(ns), FAKE, 1 << 30, None) == mu.ERR_DTYPE
    m = (mu.Matrix * 1)(mu.Matrix(FAKE, FAKE, FAKE, None, 32, 64))
    assert L.muon_step(m, 1, C.byref(mu.step_params(ns=ns)), FAKE, 1 << 30, None) == mu.ERR_DTYPE


def test_workspace_covers_both_planes(L):
    one, two = mu.stack_params(ns=mu.ns_params(compute=mu.F16)), mu.stack_params(ns=mu.ns_params(compute=mu.F16X2))
    s = stack(rows=256, cols=512, count=8)
    X, A = 8 * 256 * 512 * 2, 8 * 256 * 256 * 2
    assert L.muon_stack_workspace_size(s, 1, C.byref(two)) >= 2 * (2 * X + 2 * A)
    assert L.muon_stack_workspace_size(s, 1, C.byref(one)) >= 2 * X + 2 * A


def test_struct_layout_matches_c(tmp_path):
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "muon.h"\nint main(void){printf("%zu %zu %zu %zu %zu %zu\\n",'
                   "sizeof(muon_stack), offsetof(muon_stack, count), offsetof(muon_stack, copy_ld), sizeof(muon_stack_params),"
                   "offsetof(muon_stack_params, ns), offsetof(muon_stack_params, dev_status));return 0;}\n")
    subprocess.run(["gcc", "-I", inc, str(src), "-o", str(tmp_path / "s")], check=True)
    got = list(map(int, subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()))
    assert got == [C.sizeof(mu.StackArray), mu.StackArray.count.offset, mu.StackArray.copy_ld.offset, C.sizeof(mu.StackParams),
                   mu.StackParams.ns.offset, mu.StackParams.dev_status.offset]


def test_binding_refuses_wrong_tensors(L):
    W, M = torch.zeros(2, 8, 16), torch.zeros(2, 8, 16)
    p = mu.stack_params()
    cases = [
        (lambda: mu.StackStep([mu.Stack(W, M)], p), mu.ERR_INVALID_ARG),  # not on a GPU
        (lambda: mu.StackStep([mu.Stack(W[0], M[0])], p), mu.ERR_SHAPE),
        (lambda: mu.StackStep([mu.Stack(W, M[:1])], p), mu.ERR_SHAPE),
        (lambda: mu.StackStep([mu.Stack(W, M, M.mT)], p), mu.ERR_SHAPE),
        (lambda: mu.StackStep([mu.Stack(W.mT, M.mT)], p), mu.ERR_SHAPE),
        (lambda: mu.StackStep([mu.Stack(W, M.half())], p), mu.ERR_DTYPE),
    ]
    for i, (f, code) in enumerate(cases):
        with pytest.raises(mu.MuonError) as err:
            f()
        assert err.value.code == code, i


def test_status_words_and_workspaces_elsewhere_are_refused(L):
    """The kernels write to both: memory of the host, of another type or in pieces is refused before any launch."""
    for word in (torch.zeros(1, dtype=torch.int32), torch.zeros(1)):
        with pytest.raises(mu.MuonError) as err:
            mu.stack_params(dev_status=word)
        assert err.value.code == mu.ERR_INVALID_ARG
    for device, ws in ((0, torch.zeros(64, dtype=torch.uint8)), (-1, torch.zeros(8, 8, dtype=torch.uint8)[:, :4])):
        with pytest.raises(mu.MuonError) as err:
            mu._ws_bytes(ws, device, "here")
        assert err.value.code == mu.ERR_INVALID_ARG
    assert mu._ws_bytes(torch.zeros(8, 8), -1, "here") == 256


def test_clusters_that_cannot_run_are_left_out(tmp_path):
    """A device (or a part of one) that holds no cluster of 16, or of any size: the stack goes to a smaller cluster or to
    the chain of launches; on a whole B200 the choice is the measured one."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(mu.__file__))), "newton_schulz_10_b200", "csrc")
    src = tmp_path / "m.cpp"
    src.write_text('#include <stdio.h>\n#include "resident_model.h"\n'
                   "int main(){const int most[]={16,8,4,1};const int64_t s[][3]={{1,128,2048},{12,64,768},{1,128,128},{16,128,512}};\n"
                   "for(auto& k:s)for(int m:most){int c=-1;const bool fits=muon::res::choose_cluster(k[1],k[2],k[0],5,2,"
                   "[m](int C){return C<=m?148/C:0;},&c);printf(\"%d %d \",(int)fits,c);}return 0;}\n")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(tmp_path / "m")], check=True)
    got = list(map(int, subprocess.run([str(tmp_path / "m")], capture_output=True, text=True, check=True).stdout.split()))
    choice = list(zip(got[::2], got[1::2]))
    assert choice[:4] == [(1, 16), (0, 0), (0, 0), (0, 0)]  # 128 x 2048 fits 16 CTAs only
    assert choice[4] == choice[5] == (1, 8) and choice[6] == (1, 4)  # 64 x 768
    assert choice[8:12] == [(1, 1)] * 4  # 128 x 128
    assert choice[12][0] == choice[13][0] == choice[14][0] == 1 and all(c <= 4 for _, c in choice[14:16])
