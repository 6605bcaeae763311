"""The training operators' C entry points check their arguments on the host.

Runs without a GPU: every call here is refused before any CUDA call.
"""

import ctypes as C

import pytest

from speculative_decoding_head_gb300 import binding, build

EINVAL = 1
OK = C.c_void_p(256)     # never dereferenced: the checks come first
ODD = C.c_void_p(264)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _lce(**kw):
    a = {**dict(N=8, K=16, V=32, layout=0, ldx=16, ldw=16, ldu=32, lddx=16, lddw=16), **kw}
    return binding.LceDims(*(a[f] for f, _ in binding.LceDims._fields_))


def test_linear_ce_arguments(lib):
    def fwd(d, **kw):
        a = {**dict(X=OK, W=OK, U=OK, t=OK, loss=OK, lse=OK, scratch=OK, st=OK), **kw}
        return lib.dspark_linear_ce(C.byref(d) if d else None, a["X"], a["W"], a["U"], a["t"], a["loss"], a["lse"],
                                    a["scratch"], a["st"], None)

    def grad(d, **kw):
        a = {**dict(X=OK, W=OK, U=OK, t=OK, lse=OK, wt=OK, dX=OK, dW=OK, scratch=OK, st=OK), **kw}
        return lib.dspark_linear_ce_grad(C.byref(d) if d else None, a["X"], a["W"], a["U"], a["t"], a["lse"], a["wt"],
                                         1.0, a["dX"], a["dW"], a["scratch"], a["st"], None)

    bad_dims = [dict(N=-1), dict(K=0), dict(V=0), dict(layout=2), dict(N=(1 << 20) + 1), dict(K=65537),
                dict(V=(1 << 24) + 1), dict(ldx=15), dict(ldx=20), dict(ldw=8), dict(ldu=31), dict(ldu=34),
                dict(layout=1, ldw=24)]
    for kw in bad_dims:
        assert fwd(_lce(**kw)) == EINVAL, kw
        assert grad(_lce(**kw)) == EINVAL, kw
    assert fwd(None) == EINVAL and grad(None) == EINVAL
    for name in ("X", "W", "t", "loss", "lse", "scratch", "st"):
        assert fwd(_lce(), **{name: None}) == EINVAL, name
    for name in ("X", "W", "U", "t", "loss", "lse", "scratch"):
        assert fwd(_lce(), **{name: ODD}) == EINVAL, name
    for name in ("X", "W", "t", "lse", "scratch", "st"):
        assert grad(_lce(), **{name: None}) == EINVAL, name
    for name in ("X", "W", "U", "t", "lse", "wt", "dX", "dW", "scratch"):
        assert grad(_lce(), **{name: ODD}) == EINVAL, name
    assert grad(_lce(), dX=None, dW=None) == EINVAL
    assert grad(_lce(lddx=12)) == EINVAL and grad(_lce(lddw=12)) == EINVAL
    assert lib.dspark_linear_ce_scratch_bytes(None) == 0
    assert lib.dspark_linear_ce_scratch_bytes(C.byref(_lce(K=0))) == 0
    # the scratch grows with the rows, not with rows x vocabulary
    small = lib.dspark_linear_ce_scratch_bytes(C.byref(_lce(N=4096, K=256, V=129280)))
    assert 0 < small < 4096 * 129280 * 2
