"""Host-side checks of include/fa_rope.h and include/fa_cache.h: exports, the
refusals of every entry point (all before any CUDA call), the bindings'
argument checks, and the fp64 definitions against hand-worked values.  No
kernel runs here."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from tiled_attention_16_b200 import attention as A
from tiled_attention_16_b200 import cache, rope
from tiled_attention_16_b200.build import build

build()
P = 0x10000   # fake 256-byte aligned address; never dereferenced on rejected calls
BAD, UNSUP = A.FA_ERR_INVALID_ARG, A.FA_ERR_UNSUPPORTED


def test_exports():
    assert set(rope.declared_symbols()) == {"fa_qk_norm_rope", "fa_qk_norm_rope_bwd",
                                            "fa_qk_norm_rope_bwd_workspace_bytes"}
    assert set(cache.declared_symbols()) == {"fa_cache_write", "fa_cache_read", "fa_decode_cache",
                                             "fa_decode_cache_workspace_bytes"}
    for n in rope.declared_symbols() + cache.declared_symbols():
        assert hasattr(A.lib(), n)


def no_gpu(st):
    return st in (A.FA_ERR_CUDA, A.FA_ERR_UNSUPPORTED)


# ---- norm with rotation

def rshape(**kw):
    d = dict(B=2, Hq=4, Hkv=2, N=10, D=128, rotary_dim=128, interleaved=0, eps=1e-6, weight_bf16=0)
    d.update(kw)
    return rope.FaRopeShape(*[d[n] for n, _ in rope.FaRopeShape._fields_])


def rrows(data=P, sb=10 * 8 * 128, sh=128, sn=8 * 128):
    return rope.FaRows(data, sb, sh, sn)


def call_rope(shape=None, bwd=False, **kw):
    a = dict(q=rrows(), k=rrows(), qw=P, kw=P, f=P, pos=P, oq=P, ok=P, dq=rrows(), dk=rrows(), dqw=P, dkw=P, ws=P,
             nb=1 << 30)
    a.update(kw)
    s = rshape() if shape is None else shape
    r = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    L = rope._rope_lib()
    if not bwd:
        return L.fa_qk_norm_rope(r(s) if s else None, r(a["q"]), r(a["k"]), a["qw"], a["kw"], a["f"], a["pos"], a["oq"],
                                 a["ok"], None)
    return L.fa_qk_norm_rope_bwd(r(s) if s else None, a["oq"], a["ok"], r(a["q"]), r(a["k"]), a["qw"], a["kw"], a["f"],
                                 a["pos"], r(a["dq"]), r(a["dk"]), a["dqw"], a["dkw"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_rope_refusals(bwd):
    for kw in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(N=0), dict(D=0), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(rotary_dim=-8), dict(rotary_dim=136),
               dict(rotary_dim=12), dict(Hq=65535, Hkv=1), dict(B=1 << 16, N=1 << 16)):
        assert call_rope(rshape(**kw), bwd) == BAD, kw
        assert rope._rope_lib().fa_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(rshape(**kw))) == 0
    for d in (32, 96, 256):
        assert call_rope(rshape(D=d, rotary_dim=0), bwd) == UNSUP
    for kw in (dict(q=None), dict(k=None), dict(q=rrows(0)), dict(k=rrows(P + 8)), dict(q=rrows(sn=-8)),
               dict(q=rrows(sh=4)), dict(k=rrows(sb=12)), dict(qw=0), dict(qw=P + 2), dict(kw=P + 1), dict(f=0),
               dict(f=P + 2), dict(pos=P + 2), dict(oq=0), dict(ok=P + 8)):
        assert call_rope(bwd=bwd, **kw) == BAD, kw
    null = rope._rope_lib()
    assert null.fa_qk_norm_rope(None, None, None, P, P, P, P, P, P, None) == BAD
    assert null.fa_qk_norm_rope_bwd_workspace_bytes(None) == 0
    if not torch.cuda.is_available():
        assert no_gpu(call_rope(bwd=bwd)) and no_gpu(call_rope(rshape(rotary_dim=0), bwd, f=0, pos=0))
        # strides of dimensions of size 1 are not looked at; reads may repeat rows
        assert no_gpu(call_rope(rshape(B=1), bwd, q=rrows(sb=-3)))
        assert no_gpu(call_rope(bwd=bwd, q=rrows(sb=0, sh=0)))


def test_rope_backward_refuses_views_that_overlap():
    for kw in (dict(dq=rrows(sh=0)), dict(dq=rrows(sh=64)), dict(dk=rrows(sb=9 * 8 * 128)), dict(dk=rrows(sn=128)),
               dict(dq=None), dict(dk=rrows(P + 4)), dict(dqw=0), dict(dkw=P + 2), dict(ws=0), dict(ws=P + 16)):
        assert call_rope(bwd=True, **kw) == BAD, kw
    if not torch.cuda.is_available():
        assert no_gpu(call_rope(bwd=True, dq=rrows(sb=128 * 10 * 4, sh=128 * 10, sn=128)))


# ---- cache

def cshape(**kw):
    d = dict(B=2, Hkv=2, capacity=100, D=128, format=1)
    d.update(kw)
    return cache.FaCacheShape(*[d[n] for n, _ in cache.FaCacheShape._fields_])


def call_write(shape=None, N=10, **kw):
    a = dict(k=rrows(), v=rrows(), start=P, count=0, kc=P, vc=P, ks=P, vs=P)
    a.update(kw)
    s = cshape() if shape is None else shape
    r = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return cache._cache_lib().fa_cache_write(r(s), N, r(a["k"]), r(a["v"]), a["start"], a["count"], a["kc"], a["vc"],
                                             a["ks"], a["vs"], None)


def call_read(shape=None, N=10, **kw):
    a = dict(lens=0, kc=P, vc=P, ks=P, vs=P, ok=P, ov=P)
    a.update(kw)
    s = cshape() if shape is None else shape
    return cache._cache_lib().fa_cache_read(ctypes.byref(s), N, a["lens"], a["kc"], a["vc"], a["ks"], a["vs"], a["ok"],
                                            a["ov"], None)


def test_cache_refusals():
    for f in (call_write, call_read):
        for kw in (dict(B=0), dict(Hkv=0), dict(capacity=0), dict(D=0), dict(format=-1), dict(format=3),
                   dict(capacity=102), dict(capacity=102, format=2), dict(B=1 << 15, Hkv=2)):
            assert f(cshape(**kw)) == BAD, kw
        assert f(cshape(D=96)) == UNSUP
        assert f(N=0) == BAD and f(N=-1) == BAD
        for kw in (dict(kc=0), dict(vc=P + 8), dict(ks=0), dict(vs=0), dict(ks=P + 4)):
            assert f(**kw) == BAD, kw
        if not torch.cuda.is_available():
            assert no_gpu(f()) and no_gpu(f(cshape(capacity=102, format=0), ks=0, vs=0))
    for kw in (dict(k=None), dict(v=rrows(P + 2)), dict(k=rrows(sh=-128)), dict(start=0), dict(start=P + 2),
               dict(count=P + 1)):
        assert call_write(**kw) == BAD, kw
    assert call_write(N=1 << 30) == BAD
    for kw in (dict(lens=P + 2), dict(ok=0), dict(ov=P + 8)):
        assert call_read(**kw) == BAD, kw
    assert call_read(N=101) == BAD
    assert cache._cache_lib().fa_cache_write(None, 1, None, None, P, 0, P, P, P, P, None) == BAD


def dshape(**kw):
    d = dict(B=2, Hq=8, Hkv=2, Nq=1, capacity=100, n_prefix=0, D=128, format=1, scale=0.1, causal=1)
    d.update(kw)
    return cache.FaCacheDecodeShape(*[d[n] for n, _ in cache.FaCacheDecodeShape._fields_])


def call_decode(shape=None, **kw):
    a = dict(q=P, kc=P, vc=P, ks=P, vs=P, lens=P, pk=0, pv=0, o=P, lse=P, ws=P, nb=1 << 40)
    a.update(kw)
    s = dshape() if shape is None else shape
    return cache._cache_lib().fa_decode_cache(ctypes.byref(s), a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["lens"],
                                              a["pk"], a["pv"], a["o"], a["lse"], a["ws"], a["nb"], None)


def test_decode_refusals():
    for kw in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Nq=0), dict(capacity=0), dict(capacity=101), dict(n_prefix=-1),
               dict(format=5), dict(Hq=7), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(B=1 << 15, Hkv=4), dict(B=1 << 10, Hq=1 << 10, Nq=17)):
        assert call_decode(dshape(**kw)) == BAD, kw
        assert cache._cache_lib().fa_decode_cache_workspace_bytes(ctypes.byref(dshape(**kw))) == 0
    assert call_decode(dshape(D=96)) == UNSUP
    for kw in (dict(q=0), dict(q=P + 8), dict(kc=P + 4), dict(vc=0), dict(ks=0), dict(vs=P + 8), dict(lens=0),
               dict(lens=P + 2), dict(o=0), dict(lse=0), dict(lse=P + 2)):
        assert call_decode(**kw) == BAD, kw
    for kw in (dict(ws=0), dict(ws=P + 128)):       # caches up to 512 slots without a prefix need none
        assert call_decode(dshape(capacity=516), **kw) == BAD and call_decode(dshape(n_prefix=5), pk=P, pv=P, **kw) == BAD
    assert call_decode(dshape(n_prefix=5)) == BAD and call_decode(dshape(n_prefix=5), pk=P, pv=P + 8) == BAD
    assert cache._cache_lib().fa_decode_cache_workspace_bytes(None) == 0
    if not torch.cuda.is_available():
        assert no_gpu(call_decode()) and no_gpu(call_decode(dshape(n_prefix=5), pk=P, pv=P))
        assert no_gpu(call_decode(ws=0, nb=0)) and no_gpu(call_decode(dshape(capacity=512), ws=0, nb=0))
        assert no_gpu(call_decode(dshape(format=0, capacity=101), ks=0, vs=0))


# ---- bindings

def test_bindings_check_their_tensors():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    w = torch.zeros(64)
    with pytest.raises(ValueError):
        rope.qk_norm_rope(x, x, w, w, None)          # no CPU path
    with pytest.raises(TypeError):
        rope.check_rows("x", "q", (1,))
    m = x.to("meta")
    with pytest.raises(ValueError):
        rope.qk_norm_rope(m[0], m[0], w, w, None)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        cache.cache_write(x, x, x, x, i)
    with pytest.raises(TypeError):
        cache.cache_read(x.float(), x.float())
    with pytest.raises(ValueError):
        cache.decode_cache(x, x, x, i)
    with pytest.raises(TypeError):
        cache.make_cache(1, 1, 4, 64, torch.float16, "cpu")
    k, v, ks, vs = cache.make_cache(1, 2, 8, 64, torch.int8, "cpu")
    assert k.dtype == torch.int8 and ks.shape == (1, 2, 8) and cache.make_cache(1, 1, 5, 64, device="cpu")[2] is None


# ---- the definitions

def test_rotation_by_hand():
    ang = np.array([np.pi / 2, np.pi])
    u = np.array([1.0, 2.0, 3.0, 4.0, 9.0])
    assert np.allclose(so.rotate(u, ang, False), [-3, -2, 1, -4, 9])     # pairs (0, 2), (1, 3)
    assert np.allclose(so.rotate(u, ang, True), [-2, 1, -3, -4, 9])      # pairs (0, 1), (2, 3)
    assert np.allclose(so.rotate(so.rotate(u, ang, True), ang, True, inverse=True), u)


def test_norm_by_hand():
    y, _ = so.norm_rope(np.full((1, 1, 1, 4), 3.0), np.array([1.0, 2.0, 0.5, 1.0]), np.zeros(0), np.zeros((1, 1)), 0.0, False)
    assert np.allclose(y, [[[[1.0, 2.0, 0.5, 1.0]]]])


def test_quantised_rows_by_hand():
    codes, scale = so.quantise_rows(np.array([[448.0, 17.0, -18.0, 19.0], [450.0, 1.0, 0.0, -3.0]]), "e4m3")
    assert scale.tolist() == [1.0, 2.0]
    assert codes.tolist() == [[448.0, 16.0, -18.0, 20.0], [224.0, 0.5, 0.0, -1.5]]   # 17, 19: ties to even; 225: to 224
    codes, scale = so.quantise_rows(np.array([[127.0, 2.5, -3.5, 0.5]]), "int8")
    assert scale.tolist() == [1.0] and codes.tolist() == [[127.0, 2.0, -4.0, 0.0]]
    assert np.isnan(so.quantise_rows(np.array([[np.inf, 1.0]]), "int8")[1]).all()
    assert so.quantise_rows(np.zeros((1, 4)), "e4m3")[1].tolist() == [2.0 ** -120]
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    every = every[np.isfinite(every)]
    assert (so.round_e4m3(every) == every).all()
    mid = (np.unique(every)[1:] + np.unique(every)[:-1]) / 2
    want = torch.from_numpy(mid).to(torch.float8_e4m3fn).double().numpy()
    assert (so.round_e4m3(mid) == want).all()


def test_decode_definition_agrees_with_the_attention_oracle():
    import oracle
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(2, h, n, 64, generator=g) for h, n in ((4, 3), (2, 20), (2, 20)))
    o, lse = oracle.attention_forward_kv(q, k, v, 0.2, True)
    a = so.decode_cache(q, k, v, [20, 20], 0.2, True)
    assert np.allclose(a[0], o) and np.allclose(a[1], lse)
    # the first 12 keys as a prefix, which must be the same for both sequences
    k[1, :, :12], v[1, :, :12] = k[0, :, :12], v[0, :, :12]
    o, lse = oracle.attention_forward_kv(q, k, v, 0.2, True)
    a = so.decode_cache(q, k[:, :, 12:], v[:, :, 12:], [8, 8], 0.2, True, k[0, :, :12], v[0, :, :12])
    assert np.allclose(a[0], o) and np.allclose(a[1], lse)


# ---- the headers from plain C

C_CHECK = r"""
#include <stdint.h>
#include <stdio.h>
#include "fa_cache.h"
#define CHECK(n, cond) do { if (!(cond)) { fprintf(stderr, "check %d: %s\n", n, #cond); return n; } } while (0)
int main(void) {
    void* p = (void*)(uintptr_t)0x10000;   /* never dereferenced */
    fa_rows rows = {0, 4096, 128, 512};
    fa_rope_shape rs = {1, 4, 2, 8, 96, 0, 0, 1e-6f, 0};
    fa_cache_shape cs = {1, 2, 10, 128, FA_CACHE_INT8};
    fa_cache_decode_shape ds = {1, 4, 2, 1, 12, 0, 128, FA_CACHE_E4M3, 0.0f, 1};
    rows.data = p;
    CHECK(1, fa_qk_norm_rope(&rs, &rows, &rows, p, p, 0, 0, p, p, 0) == FA_ERR_UNSUPPORTED);
    CHECK(2, fa_qk_norm_rope_bwd_workspace_bytes(&rs) == 0);
    CHECK(3, fa_qk_norm_rope_bwd(&rs, p, p, &rows, &rows, p, p, 0, 0, &rows, &rows, p, p, p, 0, 0) == FA_ERR_UNSUPPORTED);
    CHECK(4, fa_cache_write(&cs, 1, &rows, &rows, p, 0, p, p, p, p, 0) == FA_ERR_INVALID_ARG);
    CHECK(5, fa_cache_read(&cs, 1, 0, p, p, p, p, p, p, 0) == FA_ERR_INVALID_ARG);
    CHECK(6, fa_decode_cache_workspace_bytes(&ds) == 0);
    CHECK(7, fa_decode_cache(&ds, p, p, p, p, p, p, 0, 0, p, p, p, 0, 0) == FA_ERR_INVALID_ARG);
    CHECK(8, FA_CACHE_BF16 == 0 && FA_CACHE_UNDIVIDED == 512);
    printf("ok\n");
    return 0;
}
"""


def test_headers_compile_as_c99(tmp_path):
    import os
    import shutil
    import subprocess
    from tiled_attention_16_b200.build import LIB, ROOT
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    src, exe = tmp_path / "check.c", tmp_path / "check"
    src.write_text(C_CHECK)
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), LIB,
                        f"-Wl,-rpath,{os.path.dirname(LIB)}", "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr


# ---- the limits of a shape, just inside and just past each

LIMITS = [
    # rows
    (dict(B=1 << 10, Hq=1 << 10, Hkv=2, Nq=16, capacity=4), dict(B=1 << 10, Hq=(1 << 10) + 2, Hkv=2, Nq=16, capacity=4)),
    (dict(B=1, Hq=1, Hkv=1, Nq=1 << 24), dict(B=1, Hq=1, Hkv=1, Nq=(1 << 24) + 1)),
    # slots of one sequence
    (dict(B=1, Hq=1, Hkv=1, capacity=(1 << 31) - 64), dict(B=1, Hq=1, Hkv=1, capacity=(1 << 31) - 60)),
    (dict(B=1, Hq=1, Hkv=1, format=0, capacity=(1 << 31) - 64), dict(B=1, Hq=1, Hkv=1, format=0, capacity=(1 << 31) - 63)),
    # key tiles of all sequences' heads and 2 (up to 8 rows a head) or 4 for each: 65535 x 32768 is 2^31 - 32768
    (dict(B=65535, Hq=8, Hkv=1, capacity=32766 * 64), dict(B=65535, Hq=8, Hkv=1, capacity=32766 * 64 + 4)),
    (dict(B=65535, Hq=9, Hkv=1, capacity=32764 * 64), dict(B=65535, Hq=9, Hkv=1, capacity=32764 * 64 + 4)),
    # the prefix: keys, and key tiles of all heads' row tiles of 128 and of 256
    (dict(B=1, Hq=1, Hkv=1, n_prefix=(1 << 31) - 256), dict(B=1, Hq=1, Hkv=1, n_prefix=(1 << 31) - 255)),
    (dict(B=1, Hq=65535, Hkv=65535, n_prefix=32768 * 128), dict(B=1, Hq=65535, Hkv=65535, n_prefix=32768 * 128 + 1)),
    (dict(B=257, Hq=2, Hkv=1, n_prefix=(1 << 31) // 4), dict(B=257, Hq=2, Hkv=1, Nq=512, n_prefix=(1 << 31) // 4)),
    # few slots of many rows, many slots of few: no product of the two counts
    (dict(B=8, Hq=128, Hkv=1, Nq=128, D=64, capacity=1 << 20), dict(B=8, Hq=128, Hkv=1, Nq=1 << 15, D=64, capacity=1 << 20)),
    (dict(B=8, Hq=128, Hkv=1, Nq=128, n_prefix=1 << 21), dict(B=8, Hq=128, Hkv=1, Nq=128, n_prefix=1 << 30)),
]


@pytest.mark.parametrize("inside,past", LIMITS)
def test_decode_limits(inside, past):
    pre = lambda kw: dict(pk=P, pv=P) if kw.get("n_prefix") else {}  # noqa: E731
    assert call_decode(dshape(**past), **pre(past)) == BAD
    if not torch.cuda.is_available():
        assert no_gpu(call_decode(dshape(**inside), **pre(inside)))


def test_write_read_and_rope_limits():
    assert call_write(cshape(B=1, Hkv=2), N=1 << 30) == BAD and call_write(cshape(B=3, Hkv=1), N=715827883) == BAD
    assert call_rope(rshape(Hq=65535, Hkv=1)) == BAD and call_rope(rshape(B=1 << 16, N=1 << 15)) == BAD
    if not torch.cuda.is_available():
        assert no_gpu(call_write(cshape(B=1, Hkv=2), N=(1 << 30) - 1)) and no_gpu(call_write(cshape(B=3, Hkv=1), N=715827882))
        assert no_gpu(call_read(cshape(B=65535, Hkv=1, capacity=32768), N=32768))
        assert call_read(cshape(B=65535, Hkv=1, capacity=32772), N=32769) == BAD
        assert no_gpu(call_rope(rshape(Hq=65534, Hkv=1))) and no_gpu(call_rope(rshape(B=(1 << 16) - 1, N=1 << 15)))


def test_package_imports_where_torch_has_no_cuda():
    """The workloads and the oracle's users import the package on machines
    whose torch was built without CUDA, and so without these names."""
    import subprocess
    import sys
    from tiled_attention_16_b200.build import ROOT
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, n)\n"
            "import tiled_attention_16_b200 as t\n"
            "from tiled_attention_16_b200 import cache, rope, workloads\n"
            "try:\n    t.qk_norm_rope(*[torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)] * 2, *[torch.zeros(64)] * 2, None)\n"
            "except ValueError as e:\n    print('ok', e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stderr
