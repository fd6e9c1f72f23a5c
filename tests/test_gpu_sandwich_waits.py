"""A wait for a row's bulk copies that runs out, in the sandwich norm and its
gradients: everything from that row of its block on is NaN, nothing is what an
earlier row left behind.  The library is linked again with a sandwich.cu whose
waits run out after each stage's first row (native/sandwich_waits.cu); all its
copies do land."""
import subprocess
from pathlib import Path

import pytest
import torch
from test_gpu_sandwich import Grads, Made

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300 import build as build_of

pytestmark = pytest.mark.gpu
ROWS, H = 2000, 7168  # staying blocks: 304 and 152 of them
FORMS = [dict(), dict(groups=None), dict(pre=False), dict(post=False), dict(post=False, pre=False), dict(groups=[5, 700, 700, 1990])]


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    """A library whose waits run out, with binding's signatures."""
    import ctypes
    build_of.build()
    if not (build_of.BUILD / "sandwich.o").exists():
        build_of.build(force=True)
    at = tmp_path_factory.mktemp("late")
    src = Path(__file__).parent / "native" / "sandwich_waits.cu"
    include = [a for p in (build_of.CSRC, build_of.PKG.parent / "include") for a in ("-I", str(p))]
    subprocess.run([build_of.nvcc(), *build_of.ARCH, *build_of.FLAGS, *include, "-c", str(src), "-o", str(at / "late.o")], check=True)
    objects = [build_of.BUILD / (Path(s).stem + ".o") for s in build_of.SOURCES if s != "sandwich.cu"]
    subprocess.run([build_of.nvcc(), *build_of.ARCH, "-shared", "-o", str(at / "liblate.so"), str(at / "late.o"), *map(str, objects)],
                   check=True)
    lib = ctypes.CDLL(str(at / "liblate.so"))
    for name, restype, argtypes in B.SIGNATURES:
        f = getattr(lib, name)
        f.restype, f.argtypes = restype, argtypes
    return lib


def blocks_rows(rows, blocks, stages):
    """(rows that each block sees, rows from which on it sees none), as masks."""
    chunk = -(-rows // blocks)
    at = torch.arange(rows, device="cuda") % chunk
    return at < stages, at >= stages


def check(name, got, want, inside, blocks, stages):
    """Rows of a stage's first use are right, the others NaN; those in no group
    as they were."""
    right, gone = blocks_rows(ROWS, blocks, stages)
    a, b = got.view(torch.uint8).view(ROWS, -1), want.view(torch.uint8).view(ROWS, -1)
    assert torch.equal(a[right | ~inside], b[right | ~inside]), name
    assert torch.isnan(got.float()[gone & inside]).all(), name


@pytest.mark.parametrize("form", FORMS, ids=str)
def test_norm(late, form, monkeypatch):
    m = Made(ROWS, H, **form)
    for kept in (False, True):
        want = m.forward(kept=kept)
        with monkeypatch.context() as c:
            c.setattr(B, "_lib", late)
            got = m.forward(kept=kept)
        for n in want:
            if n == "rstd" and None in (m.pre, m.post):
                continue  # 1 for a norm that is not there
            check(n, got[n], want[n], m.inside, 304, 3)


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_gradients(late, form, x8, monkeypatch):
    m = Made(ROWS, H, **form)
    g = Grads(m, x8, x8 and m.pre is not None)
    want = g.run()
    with monkeypatch.context() as c:
        c.setattr(B, "_lib", late)
        got = g.run()
    for n in ("dx", "dresidual"):
        check(n, got[n], want[n], m.inside, 152, 3)
    for n in set(got) - {"dx", "dresidual"}:
        sums = got[n].view(-1, H)
        empty = (want[n].view(-1, H) == 0).all(1)  # a group without rows
        assert torch.isnan(sums[~empty]).all() and (sums[empty] == 0).all(), n
