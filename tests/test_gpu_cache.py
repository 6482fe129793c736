"""GPU parity of cache_write, cache_read and decode_cache against the fp64
definitions.

Codes and scales have to be equal to the definition's.  Decoding, from the
arithmetic: P is rounded to bf16 (2^-8 of each weight; bf16 cache or prefix) or
fp16 (2^-11), so O moves by at most that times sum_j p_j |v_j|; a score is a
sum of D products in fp32, off by at most (D + 16) 2^-23 of its largest sum of
magnitudes, which moves every weight by that (twice: numerator and sum); the
exponentials and the fp32 sums add 2^-18; the result is rounded to bf16 (2^-8).
8-bit caches: a weight times its V scale, the row's largest weight at 2^6 or more
and the scale over a power of two below twice the largest, is subnormal in fp16
below 2^-14 and then off by up to 2^-25, so each key may add 2^-25 / 2^6 * 2 =
2^-30 of the largest |scale * code| there is.
"""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from tiled_attention_16_b200 import attention as A
from tiled_attention_16_b200 import cache, rope

pytestmark = pytest.mark.gpu

BF = torch.finfo(torch.bfloat16).eps / 2
FMT = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def np64(t):
    return t.detach().double().cpu().numpy()


def values(codes, scale):
    return np64(codes) if scale is None else np64(codes) * np64(scale)[..., None]


def new_cache(B, H, cap, D, fmt, dev, fill=True):
    k, v, ks, vs = cache.make_cache(B, H, cap, D, FMT[fmt], dev)
    if fill:   # bytes that are NaN as e4m3 and as bf16, NaN scales: nothing may read them
        for t in (k, v):
            t.view(torch.uint8).fill_(0xFF)
        for t in (ks, vs):
            if t is not None:
                t.fill_(float("nan"))
    return k, v, ks, vs


def rows(B, H, N, D, seed, token_major=False, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    shape = (B, N, H, D) if token_major else (B, H, N, D)
    x = (sigma * torch.randn(shape, generator=g)).to(torch.bfloat16).to(_gpu())
    return x.transpose(1, 2) if token_major else x


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=_gpu())


# ---------------------------------------------------------------- write, read

@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("B,H,N,cap,D", [(1, 1, 1, 4, 128), (3, 2, 5, 64, 64), (2, 3, 67, 132, 128), (4, 8, 33, 40, 64),
                                         (2, 40, 1, 8, 128), (1, 100, 1, 4, 64), (2, 33, 3, 12, 128), (1, 17, 130, 200, 64)])
def test_write_then_read(fmt, B, H, N, cap, D):
    dev = _gpu()
    kc, vc, ks, vs = new_cache(B, H, cap, D, fmt, dev)
    before = [t.clone() for t in (kc, vc)]
    k, v = rows(B, H, N, D, 1, sigma=3.0), rows(B, H, N, D, 2, token_major=True, sigma=0.01)
    start = ints(*[(7 * b) % max(1, cap - N + 1) for b in range(B)])
    cache.cache_write(k, v, kc, vc, start, k_scale=ks, v_scale=vs)
    for x, c, s, old in ((k, kc, ks, before[0]), (v, vc, vs, before[1])):
        codes, scale = (np64(x), None) if fmt == "bf16" else so.quantise_rows(np64(x), fmt)
        for b in range(B):
            at = int(start[b])
            assert (np64(c[b, :, at:at + N]) == codes[b]).all()
            if s is not None:
                assert (np64(s[b, :, at:at + N]) == scale[b]).all()
                assert torch.isnan(s[b, :, :at]).all() and torch.isnan(s[b, :, at + N:]).all()
            keep = torch.ones(cap, dtype=torch.bool)
            keep[at:at + N] = False
            assert torch.equal(c[b].view(torch.uint8)[:, keep], old[b].view(torch.uint8)[:, keep])
    lens = start + N
    n = int(lens.max())
    rk, rv = cache.cache_read(kc[:, :, :], vc, n, lens=lens, k_scale=ks, v_scale=vs)
    for x, r, f in ((k, rk, ks), (v, rv, vs)):
        codes, scale = (np64(x), np.ones(x.shape[:3])) if fmt == "bf16" else so.quantise_rows(np64(x), fmt)
        for b in range(B):
            at = int(start[b])
            want = codes[b] * scale[b][..., None]
            got = np64(r[b, :, at:at + N])
            # e4m3 values times a power of two are bf16 numbers; int8 ones are rounded (in fp32, then bf16)
            tol = BF * (1 + 2.0 ** -14) * np.abs(want) if fmt == "int8" else 0.0
            assert (np.abs(got - want) <= tol).all()
            assert (r[b, :, at + N:] == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rounding_over_the_whole_range(fmt):
    """Rows of every magnitude a bf16 has, ties between codes, largest values at
    and around the steps of the scale."""
    dev = _gpu()
    D, N = 128, 600
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, 1, N, D, generator=g) * torch.exp2(torch.linspace(-132, 120, N))[None, None, :, None]
    x[0, 0, 0] = 0
    x[0, 0, 1] = torch.arange(D).float() * 2.0 ** -133                    # subnormal
    x[0, 0, 2, 0], x[0, 0, 2, 1:] = 3.38e38, 1.0
    for i, top in enumerate((448.0, 450.0, 446.0, 447.0, 224.0, 1.75, 1.7578125, 127.0, 254.0, 63.5)):
        x[0, 0, 10 + i] = torch.linspace(-1, 1, D) * top
        x[0, 0, 10 + i, 0] = top
    x[0, 0, 30] = (torch.arange(D) - 64).float() + 0.5                    # ties of int8 under a scale of 1 (amax 127)
    x[0, 0, 30, 0] = 127.0
    x[0, 0, 31] = torch.arange(D).float() * 2.0 ** -4 + 16                # ties of e4m3
    x = x.to(torch.bfloat16).to(dev)
    kc, vc, ks, vs = new_cache(1, 1, N, D, fmt, dev)
    cache.cache_write(x, x, kc, vc, ints(0), k_scale=ks, v_scale=vs)
    codes, scale = so.quantise_rows(np64(x), fmt)
    assert (np64(ks) == scale).all()
    assert (np64(kc) == codes).all()
    assert torch.equal(kc.view(torch.uint8), vc.view(torch.uint8)) and torch.equal(ks, vs)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rows_with_infinities_and_nans_read_back_as_nan(fmt):
    dev = _gpu()
    x = rows(1, 2, 6, 64, 9).clone()
    x[0, 0, 1, 3] = float("inf")
    x[0, 1, 2, 63] = float("nan")
    x[0, 1, 4, 0] = -float("inf")
    kc, vc, ks, vs = new_cache(1, 2, 8, 64, fmt, dev)
    cache.cache_write(x, x, kc, vc, ints(1), k_scale=ks, v_scale=vs)
    k, _ = cache.cache_read(kc, vc, 7, lens=ints(7), k_scale=ks, v_scale=vs)
    bad = torch.zeros(2, 6, dtype=torch.bool, device=dev)
    bad[0, 1] = bad[1, 2] = bad[1, 4] = True
    assert torch.isnan(k[0, :, 1:][bad]).all() and torch.isfinite(k[0, :, 1:][~bad]).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_rows_without_a_slot_are_dropped(fmt):
    """Negative starts, starts behind the end, counts below N, 0 and above N."""
    dev = _gpu()
    B, H, N, cap, D = 6, 2, 5, 12, 64
    start, count = ints(-2, 10, 2 ** 31 - 2, -(2 ** 31), 3, 0), ints(5, 9, 5, 5, 2, 0)
    kc, vc, ks, vs = new_cache(B, H, cap, D, fmt, dev)
    k, v = rows(B, H, N, D, 3), rows(B, H, N, D, 4)
    cache.cache_write(k, v, kc, vc, start, count, ks, vs)
    written = torch.zeros(B, cap, dtype=torch.bool)
    for b in range(B):
        for n in range(min(N, int(count[b]))):
            if 0 <= int(start[b]) + n < cap:
                written[b, int(start[b]) + n] = True
    assert written.sum() == 3 + 2 + 2
    clean = (kc.view(torch.uint8) != 0xFF).any(-1)[:, 0].cpu()
    assert torch.equal(clean, written)
    ref = np64(k[0, :, 2:]) if fmt == "bf16" else so.quantise_rows(np64(k[0, :, 2:]), fmt)[0]
    assert (np64(kc[0, :, :3]) == ref).all()


def test_captured_write_follows_the_device_lengths():
    dev = _gpu()
    kc, vc, ks, vs = new_cache(2, 2, 16, 128, "e4m3", dev)
    k, v = rows(2, 2, 1, 128, 1), rows(2, 2, 1, 128, 2)
    start = ints(0, 3)
    q = rows(2, 4, 1, 128, 3)
    cache.cache_write(k, v, kc, vc, start, k_scale=ks, v_scale=vs)
    vc[1, :, :3], kc[1, :, :3] = 0, 0
    ks[1, :, :3], vs[1, :, :3] = 1, 1
    assert cache.decode_cache_workspace_bytes(2, 4, 2, 1, 16, 128, torch.float8_e4m3fn) == 0
    cache.decode_cache(q, kc, vc, start + 1, ks, vs)
    torch.cuda.synchronize()
    lens = start + 1
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.cache_write(k, v, kc, vc, start, k_scale=ks, v_scale=vs)
        o, lse = cache.decode_cache(q, kc, vc, lens, ks, vs)
        start += 1
        lens += 1
    for step in range(5):
        k.copy_(rows(2, 2, 1, 128, 10 + step))
        v.copy_(rows(2, 2, 1, 128, 20 + step))
        n = lens.clone()
        g.replay()
        torch.cuda.synchronize()
        want = cache.decode_cache(q, kc, vc, n, ks, vs)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        check_decode(q, kc, vc, ks, vs, n, (o, lse))
    assert start.tolist() == [5, 8]


# ---------------------------------------------------------------- decoding

def lens_mask(lens, shape):
    """Which of [B, H, cap, D] lie below the lengths."""
    return np.broadcast_to((np.arange(shape[2]) < lens.cpu().numpy()[:, None])[:, None, :, None], shape)


def check_decode(q, kc, vc, ks, vs, lens, got, causal=True, scale=None, pk=None, pv=None):
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    k, v = values(kc, ks), values(vc, vs)
    for b in range(q.shape[0]):   # what lies behind a length is anything
        n = min(max(int(lens[b]), 0), k.shape[2])
        k[b, :, n:], v[b, :, n:] = 0, 0
    o, lse, wt, size = so.decode_cache(np64(q), k, v, lens.tolist(), scale, causal,
                                       None if pk is None else np64(pk), None if pv is None else np64(pv))
    u = BF if ks is None or pk is not None else 2.0 ** -11
    ds = (D + 16) * 2.0 ** -23 * size
    go, gl = np64(got[0]), np64(got[1])
    assert (np.isneginf(gl) == np.isneginf(lse)).all() and (go[np.isneginf(lse)] == 0).all()
    some = ~np.isneginf(lse)
    tol = (u * 1.01 + 2 * ds + 2.0 ** -18)[..., None] * wt + BF * 1.01 * np.abs(o)
    if ks is not None:
        top = np.repeat(np.abs(values(vc, vs)).max((2, 3), initial=0.0, where=lens_mask(lens, v.shape)), q.shape[1] // v.shape[1], 1)
        tol = tol + (2.0 ** -30 * top * np.clip(lens.cpu().numpy(), 0, v.shape[2])[:, None])[..., None, None]
    err = np.abs(go - o)
    assert (err[some] <= tol[some]).all(), f"O off by {(err[some] / tol[some]).max()} of its tolerance"
    tl = ds + 2.0 ** -18 + 2.0 ** -22 * np.abs(np.where(some, lse, 0))
    assert (np.abs(gl - np.where(some, lse, 0))[some] <= tl[some]).all()


def filled(B, H, cap, D, fmt, lens, dev, seed=1, sk=1.0, sv=1.0):
    """A cache whose slots below each length were written; the rest is NaN."""
    kc, vc, ks, vs = new_cache(B, H, cap, D, fmt, dev)
    n = max(1, min(cap, max(lens)))
    k, v = rows(B, H, n, D, seed, sigma=sk), rows(B, H, n, D, seed + 1, sigma=sv)
    cache.cache_write(k, v, kc, vc, ints(*[0] * B), ints(*[max(0, x) for x in lens]), ks, vs)
    return kc, vc, ks, vs


DECODE = [
    # B, Hq, Hkv, Nq, cap, D, lens, causal
    (1, 1, 1, 1, 4, 128, [1], True),
    (1, 2, 1, 1, 64, 64, [64], True),
    (2, 8, 2, 1, 300, 128, [300, 65], True),
    (3, 4, 4, 1, 200, 64, [0, 1, 200], True),              # an empty sequence
    (2, 8, 1, 3, 132, 128, [131, 2], True),                # 24 rows: two row blocks; a row before the first key
    (2, 12, 4, 5, 260, 64, [3, 259], False),
    (5, 8, 8, 2, 1000, 128, [17, 1000, 63, 64, 641], True),
    (1, 40, 8, 1, 2500, 128, [2497], True),
    (40, 4, 2, 1, 96, 64, [(7 * b) % 97 for b in range(40)], True),
    (1, 16, 1, 4, 20000, 128, [19999], True),              # 64 rows of one head, many shares of a unit
    (700, 2, 2, 1, 68, 64, [(5 * b) % 69 for b in range(700)], True),   # more units than CTAs
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,cap,D,lens,causal", DECODE)
def test_decode_ragged(fmt, B, Hq, Hkv, Nq, cap, D, lens, causal):
    dev = _gpu()
    kc, vc, ks, vs = filled(B, Hkv, cap, D, fmt, lens, dev)
    q = rows(B, Hq, Nq, D, 77)
    got = cache.decode_cache(q, kc, vc, ints(*lens), ks, vs, causal=causal)
    assert A.device_status(dev) == A.FA_OK, f"sites {A.timeout_sites():#x}"
    check_decode(q, kc, vc, ks, vs, ints(*lens), got, causal)


PREFIX = [
    # B, Hq, Hkv, Nq, cap, D, Np, lens
    (1, 1, 1, 1, 4, 128, 1, [1]),
    (2, 8, 2, 1, 64, 128, 127, [0, 64]),
    (3, 4, 2, 2, 100, 64, 128, [100, 5, 1]),
    (16, 8, 1, 1, 64, 128, 1000, list(range(16))),           # 128 rows: one tile, alternating blocks
    (17, 8, 1, 1, 64, 128, 385, [64 - b for b in range(17)]),   # 136 rows: two tiles share the keys
    (33, 8, 2, 2, 32, 64, 700, [b % 33 for b in range(33)]),    # 264 rows: three tiles, the last nearly empty
    (4, 32, 8, 1, 132, 128, 4100, [1, 130, 50, 90]),
    (2, 2, 1, 1, 64, 64, 40000, [64, 0]),
    (1, 100, 100, 1, 4, 64, 2600, [3]),                         # one row tile each: CTAs begin and end inside heads
    (130, 16, 16, 1, 4, 128, 2000, [b % 5 for b in range(130)]),   # the same with two
    (300, 64, 32, 2, 4, 64, 200, [1] * 300),                    # more (head, row tile) pairs than CTAs
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,cap,D,Np,lens", PREFIX)
def test_decode_behind_a_prefix(fmt, B, Hq, Hkv, Nq, cap, D, Np, lens):
    dev = _gpu()
    kc, vc, ks, vs = filled(B, Hkv, cap, D, fmt, lens, dev, seed=31)
    q = rows(B, Hq, Nq, D, 78)
    pk, pv = rows(1, Hkv, Np, D, 5)[0].contiguous(), rows(1, Hkv, Np, D, 6)[0].contiguous()
    got = cache.decode_cache(q, kc, vc, ints(*lens), ks, vs, pk, pv)
    assert A.device_status(dev) == A.FA_OK, f"sites {A.timeout_sites():#x}"
    check_decode(q, kc, vc, ks, vs, ints(*lens), got, pk=pk, pv=pv)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("sk,sv,sq", [(1e-3, 1e4, 30.0), (1e4, 1e-6, 1e-4), (1.0, 1e-20, 1.0), (8.0, 1.0, 4.0)])
def test_decode_scales_of_any_size(fmt, sk, sv, sq):
    """Scales far from 1, large and tiny logits, V rows of sizes 2^40 apart."""
    dev = _gpu()
    lens = [500, 129]
    kc, vc, ks, vs = filled(2, 2, 512, 128, fmt, lens, dev, sk=sk, sv=sv)
    vs[0, 0, ::3] *= 2.0 ** 40
    q = (rows(2, 4, 1, 128, 3).float() * sq).to(torch.bfloat16)
    got = cache.decode_cache(q, kc, vc, ints(*lens), ks, vs)
    check_decode(q, kc, vc, ks, vs, ints(*lens), got)


def test_zero_queries_and_a_scale_argument():
    dev = _gpu()
    for fmt in FMT:
        kc, vc, ks, vs = filled(2, 1, 128, 64, fmt, [100, 128], dev)
        q = rows(2, 2, 1, 64, 3).clone()
        q[0] = 0
        got = cache.decode_cache(q, kc, vc, ints(100, 128), ks, vs, scale=0.37)
        check_decode(q, kc, vc, ks, vs, ints(100, 128), got, scale=0.37)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_poisoned_rows_reach_the_queries_that_see_them_only(fmt):
    dev = _gpu()
    lens = [70, 70, 70]
    kc, vc, ks, vs = filled(3, 1, 128, 64, fmt, lens, dev)
    ks[0, 0, 69] = float("nan")       # seen by the last query only
    vs[1, 0, 69] = float("nan")
    q = rows(3, 2, 2, 64, 3)
    o, lse = cache.decode_cache(q, kc, vc, ints(*lens), ks, vs)
    assert torch.isnan(o[:2, :, 1]).all() and torch.isnan(lse[0, :, 1]).all()
    assert torch.isfinite(o[:2, :, 0]).all() and torch.isfinite(o[2]).all() and torch.isfinite(lse[:, :, 0]).all()
    ks[2, 0] = float("nan")           # nothing but poison
    o, lse = cache.decode_cache(q, kc, vc, ints(*lens), ks, vs)
    assert torch.isnan(o[2]).all() and torch.isnan(lse[2]).all()


ROWS = [
    # B, Hq, Hkv, Nq, cap, D, lens, causal: query rows a K/V head from 9 to 100, around what a CTA holds
    (3, 9, 1, 1, 300, 128, [300, 1, 77], True),
    (2, 34, 2, 1, 1100, 64, [1100, 513], True),
    (2, 10, 1, 2, 1028, 128, [1, 1027], True),
    (5, 32, 1, 1, 2000, 128, [2000, 64, 65, 0, 1999], True),
    (3, 16, 2, 4, 700, 64, [700, 3, 64], True),
    (2, 33, 1, 1, 516, 128, [515, 100], False),
    (2, 20, 1, 5, 900, 64, [4, 899], True),
    (48, 8, 2, 8, 200, 128, [(11 * b) % 201 for b in range(48)], True),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,cap,D,lens,causal", ROWS)
def test_decode_many_rows_a_head(fmt, B, Hq, Hkv, Nq, cap, D, lens, causal):
    test_decode_ragged(fmt, B, Hq, Hkv, Nq, cap, D, lens, causal)


# hidden(j): keys whose score is -inf, of each sequence's own and of the prefix
MINUS_INF = [
    # B, Hq, Hkv, Nq, cap, D, Np, own, prefix
    (3, 8, 2, 1, 700, 128, 0, lambda j: j < 100, None),        # whole first tiles, a second row without them
    (3, 4, 4, 2, 300, 64, 0, lambda j: j % 3 != 1, None),
    (2, 4, 1, 1, 132, 128, 0, lambda j: j >= 0, None),         # every key
    (3, 4, 2, 1, 64, 64, 900, lambda j: j < 0, lambda j: j >= 0),              # the whole prefix, alternating blocks
    (3, 4, 2, 1, 64, 128, 900, lambda j: j < 20, lambda j: j // 128 % 2 == 0),   # one block's tiles of it
    (40, 8, 2, 1, 4, 128, 700, lambda j: j < 1, lambda j: j < 500),            # row tiles that share the keys
    (40, 8, 2, 1, 4, 64, 200, lambda j: j >= 0, lambda j: j >= 0),
]


@pytest.mark.parametrize("B,Hq,Hkv,Nq,cap,D,Np,own,prefix", MINUS_INF)
def test_scores_of_minus_infinity_are_hidden_keys(B, Hq, Hkv, Nq, cap, D, Np, own, prefix):
    """As in fa_decode.  The queries' first value is positive, and -inf in the
    keys' first place makes their scores -inf."""
    dev = _gpu()
    lens = [cap - (b % 3) for b in range(B)]
    kc, vc, _, _ = filled(B, Hkv, cap, D, "bf16", lens, dev)
    q = rows(B, Hq, Nq, D, 78)
    q[..., 0] = q[..., 0].abs() + 0.5
    mine = np.array([bool(own(j)) for j in range(cap)])
    kc[:, :, torch.from_numpy(mine).to(dev), 0] = float("-inf")
    pk = pv = None
    shared = np.zeros(0, dtype=bool)
    if Np:
        pk, pv = rows(1, Hkv, Np, D, 3)[0].contiguous(), rows(1, Hkv, Np, D, 4)[0].contiguous()
        shared = np.array([bool(prefix(j)) for j in range(Np)])
        pk[:, torch.from_numpy(shared).to(dev), 0] = float("-inf")
    o, lse = cache.decode_cache(q, kc, vc, ints(*lens), prefix_k=pk, prefix_v=pv)
    assert A.device_status(dev) == A.FA_OK, f"sites {A.timeout_sites():#x}"
    go, gl, qq, k, v = np64(o), np64(lse), np64(q), np64(kc), np64(vc)
    fk, fv = (np.zeros((Hkv, 0, D)),) * 2 if pk is None else (np64(pk), np64(pv))
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            for i in range(Nq):
                n = lens[b] - Nq + i + 1
                keep = np.concatenate([~shared, ~mine[:n]])
                ro, rl, wt, size = so.decode_rows(qq[b, h, i], np.concatenate([fk[g], k[b, g, :n]]),
                                                  np.concatenate([fv[g], v[b, g, :n]]), D ** -0.5, keep)
                if not keep.any():
                    assert np.isneginf(gl[b, h, i]) and (go[b, h, i] == 0).all()
                    continue
                ds = (D + 16) * 2.0 ** -23 * size
                tol = (BF * 1.01 + 2 * ds + 2.0 ** -18) * wt + BF * 1.01 * np.abs(ro)
                assert (np.abs(go[b, h, i] - ro) <= tol).all()
                assert abs(gl[b, h, i] - rl) <= ds + 2.0 ** -18 + 2.0 ** -22 * abs(rl)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
def test_lengths_out_of_range_are_clamped(fmt):
    dev = _gpu()
    B = 4
    kc, vc, ks, vs = filled(B, 2, 64, 64, fmt, [64] * B, dev)
    q = rows(B, 2, 1, 64, 3)
    got = cache.decode_cache(q, kc, vc, ints(-5, 1000, 2 ** 31 - 1, -(2 ** 31)), ks, vs)
    want = cache.decode_cache(q, kc, vc, ints(0, 64, 64, 0), ks, vs)
    assert A.device_status(dev) == A.FA_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (got[0][0] == 0).all() and torch.isneginf(got[1][0]).all()


def test_repeated_calls_and_streams_are_bitwise_equal():
    dev = _gpu()
    lens = ints(777, 20, 1500)
    kc, vc, ks, vs = filled(3, 2, 1504, 128, "e4m3", lens.tolist(), dev)
    q = rows(3, 8, 1, 128, 3)
    pk, pv = rows(1, 2, 900, 128, 5)[0].contiguous(), rows(1, 2, 900, 128, 6)[0].contiguous()
    want = cache.decode_cache(q, kc, vc, lens, ks, vs, pk, pv)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    res = []
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(5):
                res.append(cache.decode_cache(q, kc, vc, lens, ks, vs, pk, pv))
    torch.cuda.synchronize()
    assert all(torch.equal(r[0], want[0]) and torch.equal(r[1], want[1]) for r in res)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Np", [0, 1500])
def test_captured_calls_replay(fmt, Np):
    """A divided decode (and one behind a prefix) captured with its own
    workspace: replays follow lengths, queries and cache, and stay right when
    two graphs and eager calls are mixed."""
    dev = _gpu()
    B, Hq, Hkv, D, cap = 3, 8, 2, 128, 2000
    kc, vc, ks, vs = filled(B, Hkv, cap, D, fmt, [cap] * B, dev)
    q, lens = rows(B, Hq, 1, D, 3), ints(1, 700, 1999)
    pk, pv = ((rows(1, Hkv, Np, D, 5)[0].contiguous(), rows(1, Hkv, Np, D, 6)[0].contiguous()) if Np else (None, None))
    nbytes = cache.decode_cache_workspace_bytes(B, Hq, Hkv, 1, cap, D, FMT[fmt], Np)
    ws = torch.empty(nbytes, device=dev, dtype=torch.uint8)
    want = lambda **kw: cache.decode_cache(q, kc, vc, lens, ks, vs, pk, pv, **kw)  # noqa: E731
    a, b = want(), want(workspace=ws)
    assert nbytes > 0 and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(A.FAError):
        want(workspace=ws[256:])
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = want()
        graphs.append((g, res))
    for step in range(4):
        lens.copy_(ints(2000 - step, 64 * step, 333 * step))
        q.copy_(rows(B, Hq, 1, D, 40 + step))
        for g, res in graphs:
            g.replay()
        eager = want()
        torch.cuda.synchronize()
        for g, res in graphs:
            assert torch.equal(res[0], eager[0]) and torch.equal(res[1], eager[1])
    check_decode(q, kc, vc, ks, vs, lens, eager, pk=pk, pv=pv)


@pytest.mark.parametrize("fmt,B,Hkv,cap", [("bf16", 3, 8, 1 << 20), ("e4m3", 2, 5, 1 << 23)])
def test_offsets_past_32_bits(fmt, B, Hkv, cap):
    """Caches of more than 2^32 bytes: rows written, read and attended to at
    their far ends."""
    dev = _gpu()
    D, N, Hq = 128, 70, 2 * Hkv
    kc, vc, ks, vs = cache.make_cache(B, Hkv, cap, D, FMT[fmt], dev)
    assert kc.numel() * kc.element_size() > 1 << 32
    for t in (kc, vc):
        t.view(torch.uint8).zero_()
    for t in (ks, vs):
        if t is not None:
            t.fill_(1.0)
    k, v = rows(B, Hkv, N, D, 1), rows(B, Hkv, N, D, 2)
    start = ints(*[cap - N - 3 * b for b in range(B)])
    cache.cache_write(k, v, kc, vc, start, k_scale=ks, v_scale=vs)
    b, h = B - 1, Hkv - 1
    at = int(start[b])
    ref = np64(k[b, h]) if fmt == "bf16" else so.quantise_rows(np64(k[b, h]), fmt)[0]
    assert (np64(kc[b, h, at:at + N]) == ref).all() and not kc[b, h].view(torch.uint8)[:at].any()
    q = (4 * rows(B, Hq, 1, D, 3).float()).to(torch.bfloat16)
    lens = torch.zeros_like(start)
    lens[b] = start[b] + N
    o, lse = cache.decode_cache(q, kc, vc, lens, ks, vs)
    assert A.device_status(dev) == A.FA_OK
    # keys before `at` are zero: each has the score 0 and the value 0
    kk, vv = (np64(c[b, :, at:at + N]) * (1 if s is None else np64(s[b, :, at:at + N])[..., None])
              for c, s in ((kc, ks), (vc, vs)))
    for head in (0, Hq - 1):
        s = kk[head // 2] @ np64(q[b, head, 0]) * D ** -0.5
        total = np.log(at + np.exp(s).sum())
        ref = np.exp(s - total) @ vv[head // 2]
        assert abs(float(lse[b, head, 0]) - total) <= 1e-4
        wt = np.exp(s - total) @ np.abs(vv[head // 2])
        assert (np.abs(np64(o[b, head, 0]) - ref) <= 1e-2 * wt + 1e-6).all()
    assert torch.isneginf(lse[0]).all() and (o[0] == 0).all()
    del kc, vc, ks, vs
    torch.cuda.empty_cache()


def test_refusals_on_the_gpu():
    """What only the binding or a device pointer can show wrong."""
    dev = _gpu()
    kc, vc, ks, vs = filled(1, 1, 64, 64, "int8", [64], dev)
    q, lens, k = rows(1, 1, 1, 64, 3), ints(64), rows(1, 1, 1, 64, 4)
    for bad in (dict(k_scale=None), dict(v_scale=ks.double()), dict(workspace=torch.empty(1, device=dev).expand(1 << 30)),
                dict(prefix_k=k[0], prefix_v=k[0], workspace=torch.empty(8, device=dev)), dict(prefix_k=k[0]), dict(scale=-1.0), dict(lse=ks),
                dict(out=q.transpose(0, 1)[:, :, :, :32]), dict(prefix_k=k[0], prefix_v=k[0, :, :, :32])):
        with pytest.raises((TypeError, ValueError, A.FAError)):
            cache.decode_cache(q, kc, vc, lens, **{**dict(k_scale=ks, v_scale=vs), **bad})
    for args in ((q.float(), kc, vc, lens), (q, kc.float(), vc, lens), (q, kc, vc[:, :, :32], lens),
                 (q, kc, vc, lens.long()), (q[..., ::2], kc, vc, lens), (q, kc, vc, lens.cpu())):
        with pytest.raises((TypeError, ValueError, A.FAError)):
            cache.decode_cache(*args, k_scale=ks, v_scale=vs)
    for args in ((k.float(), k), (k[..., ::2], k), (k, k[:, :, :, :32]), (k.cpu(), k)):
        with pytest.raises((TypeError, ValueError, A.FAError)):
            cache.cache_write(*args, kc, vc, lens, k_scale=ks, v_scale=vs)
    with pytest.raises(A.FAError):
        cache.cache_write(torch.empty(1, 1, 1, 68, device=dev, dtype=torch.bfloat16)[..., 4:], k, kc, vc, lens,
                          k_scale=ks, v_scale=vs)       # 8-byte aligned
    with pytest.raises(A.FAError):
        cache.cache_read(kc, vc, 65, k_scale=ks, v_scale=vs)
    cache.cache_write(k[:, :, :0], k[:, :, :0], kc, vc, lens, k_scale=ks, v_scale=vs)   # nothing to write
    assert A.device_status(dev) == A.FA_OK


def test_refusals_of_what_is_no_tensor_and_of_too_many_rows():
    dev = _gpu()
    kc, vc, ks, vs = filled(1, 1, 64, 64, "int8", [64], dev)
    q, lens, k = rows(1, 1, 1, 64, 3), ints(64), rows(1, 1, 1, 64, 4)
    for args, more in (((None, kc, vc, lens), {}), ((q, None, vc, lens), {}), ((q, kc, None, lens), {}),
                       ((q, kc, vc, None), {}), ((q, kc, vc, [64]), {}), ((q, kc, vc, lens), dict(workspace=7)),
                       ((q, kc, vc, lens), dict(prefix_k=[1], prefix_v=[1]))):
        with pytest.raises((TypeError, ValueError)):
            cache.decode_cache(*args, **{**dict(k_scale=ks, v_scale=vs), **more})
    many = k.expand(1, 1, 2 ** 32 + 1, 64)       # wraps to one row in 32 bits
    for args in ((None, k, kc, vc, lens), (k, None, kc, vc, lens), (many, many, kc, vc, lens)):
        with pytest.raises((TypeError, ValueError)):
            cache.cache_write(*args, k_scale=ks, v_scale=vs)
    assert A.device_status(dev) == A.FA_OK


def test_bf16_cache_agrees_with_decode():
    """Full lengths: the same attention as decode over the same history."""
    dev = _gpu()
    k, v, q = rows(2, 2, 640, 128, 1), rows(2, 2, 640, 128, 2), rows(2, 8, 3, 128, 3)
    a = A.decode(q, k, v, causal=True)
    b = cache.decode_cache(q, k, v, ints(640, 640))
    assert (a[0].float() - b[0].float()).abs().max() <= 2e-2 and (a[1] - b[1]).abs().max() <= 1e-3


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
def test_prefix_equals_a_copy_in_every_cache(fmt):
    """A shared prefix gives what a copy of it in front of each sequence's own
    rows gives (bf16 caches: the same numbers go in)."""
    dev = _gpu()
    B, Hq, Hkv, D, Np, n = 3, 6, 2, 64, 200, 50
    pk, pv = rows(1, Hkv, Np, D, 5), rows(1, Hkv, Np, D, 6)
    k, v, q = rows(B, Hkv, n, D, 7), rows(B, Hkv, n, D, 8), rows(B, Hq, 2, D, 9)
    own = new_cache(B, Hkv, 64, D, fmt, dev)
    cache.cache_write(k, v, own[0], own[1], ints(0, 0, 0), k_scale=own[2], v_scale=own[3])
    a = cache.decode_cache(q, own[0], own[1], ints(n, n, n), own[2], own[3], pk[0].contiguous(), pv[0].contiguous())
    back = cache.cache_read(own[0], own[1], n, k_scale=own[2], v_scale=own[3])
    both = [torch.cat([p.expand(B, -1, -1, -1), x], 2).contiguous() for p, x in zip((pk, pv), back)]
    b = cache.decode_cache(q, both[0], both[1], ints(*[Np + n] * 3))
    assert (a[0].float() - b[0].float()).abs().max() <= 2e-2 and (a[1] - b[1]).abs().max() <= 2e-3


def test_tokens_through_norm_cache_and_decoding():
    """Serving as it is used: the prompt goes through qk_norm_rope and fwd and
    into an 8-bit cache; each new token through qk_norm_rope, cache_write and
    decode_cache behind a shared prefix; the history reads back."""
    dev = _gpu()
    B, Hq, Hkv, D, Np, N = 2, 4, 2, 128, 150, 70
    g = torch.Generator().manual_seed(4)
    w = [(1 + 0.1 * torch.randn(D, generator=g)).to(dev) for _ in range(2)]
    inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(dev)

    def project(b, n):
        x = torch.randn(b, n, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).to(dev).transpose(1, 2)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    def place(b, n, at):
        return (torch.arange(n, dtype=torch.int32)[None] + at).expand(b, n).contiguous().to(dev)

    _, pk, pv = project(1, Np)
    pk = rope.qk_norm_rope(pk, pk, w[1], w[1], inv, positions=place(1, Np, 0))[0][0]
    pv = pv[0].contiguous()
    kc, vc, ks, vs = new_cache(B, Hkv, 128, D, "e4m3", dev)
    lens = ints(0, 0)
    for at, n in ((0, N), (N, 1), (N + 1, 1), (N + 2, 3)):
        q, k, v = project(B, n)
        q, k = rope.qk_norm_rope(q, k, w[0], w[1], inv, positions=place(B, n, Np + at))
        cache.cache_write(k, v, kc, vc, lens, k_scale=ks, v_scale=vs)
        lens = lens + n
        got = cache.decode_cache(q, kc, vc, lens, ks, vs, pk, pv)
        assert A.device_status(dev) == A.FA_OK
        check_decode(q, kc, vc, ks, vs, lens, got, pk=pk, pv=pv)
    hk, hv = cache.cache_read(kc, vc, int(lens[0]), lens=lens, k_scale=ks, v_scale=vs)
    assert (np64(hk) == values(kc, ks)[:, :, :int(lens[0])]).all()
    o, lse = A.fwd(hk, hk, hv, causal=True)     # the history as the next chunk's forward takes it
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


POISON = [
    # B, Hq, Hkv, Nq, cap, D, Np, lens: rows a K/V head in one block of 8, 16, 32 and several; hidden keys in one tile and in more
    (2, 2, 1, 2, 128, 64, 0, [70, 64]),
    (2, 8, 2, 3, 200, 128, 0, [65, 130]),
    (2, 8, 2, 5, 1400, 128, 0, [1398, 3]),
    (1, 2, 1, 70, 700, 64, 0, [650]),
    (2, 1, 1, 100, 128, 128, 0, [128, 60]),
    (2, 4, 2, 4, 700, 64, 300, [699, 2]),
]


@pytest.mark.parametrize("B,Hq,Hkv,Nq,cap,D,Np,lens", POISON)
def test_poisoned_bf16_values_reach_the_queries_that_see_them_only(B, Hq, Hkv, Nq, cap, D, Np, lens):
    """Infinities and NaNs in some columns of V rows that the last queries see
    and the first do not: columns and queries apart from them are as without."""
    dev = _gpu()
    kc, vc, _, _ = filled(B, Hkv, cap, D, "bf16", lens, dev)
    q = rows(B, Hq, Nq, D, 41)
    pk, pv = ((rows(1, Hkv, Np, D, 5)[0].contiguous(), rows(1, Hkv, Np, D, 6)[0].contiguous()) if Np else (None, None))
    spots = {}
    for b, n in enumerate(lens):
        first = max(n - Nq + 1, 0)             # the first slot that query 0 does not see
        for slot, col, x in ((n - 1, 3, "inf"), (n - 1, D - 1, "nan"), (first, 17, "-inf"), ((first + n) // 2, 40, "nan")):
            if first <= slot < n:
                spots[b, slot, col] = float(x)
    clean = vc.clone()
    for (b, slot, col), x in spots.items():
        vc[b, :, slot, col] = x
        clean[b, :, slot] = 0
    got = cache.decode_cache(q, kc, vc, ints(*lens), prefix_k=pk, prefix_v=pv)
    want = cache.decode_cache(q, kc, clean, ints(*lens), prefix_k=pk, prefix_v=pv)
    assert A.device_status(dev) == A.FA_OK
    assert torch.equal(got[1], want[1])        # scores know nothing of V
    qq, k, v = np64(q), np64(kc), np64(vc)
    fk, fv = (np.zeros((Hkv, 0, D)),) * 2 if pk is None else (np64(pk), np64(pv))
    go = np64(got[0])
    for b, n in enumerate(lens):
        for i in range(Nq):
            end = max(n - Nq + i + 1, 0)
            seen = [s for s in spots if s[0] == b and s[1] < end]
            if not seen:
                assert torch.equal(got[0][b, :, i], want[0][b, :, i])
                continue
            for h in range(Hq):
                g = h // (Hq // Hkv)
                with np.errstate(invalid="ignore"):
                    ro, _, wt, size = so.decode_rows(qq[b, h, i], np.concatenate([fk[g], k[b, g, :end]]),
                                                     np.concatenate([fv[g], v[b, g, :end]]), D ** -0.5,
                                                     np.ones(Np + end, dtype=bool))
                # 0 * inf is no case here: no weight underflows at these logits
                assert (np.isnan(go[b, h, i]) == np.isnan(ro)).all() and (np.isinf(go[b, h, i]) == np.isinf(ro)).all()
                assert (go[b, h, i][np.isinf(ro)] == ro[np.isinf(ro)]).all()
                fin = np.isfinite(ro)
                assert fin.sum() >= D - 4
                tol = (BF * 1.01 + 2 * (D + 16) * 2.0 ** -23 * size + 2.0 ** -18) * wt[fin] + BF * 1.01 * np.abs(ro[fin])
                assert (np.abs(go[b, h, i][fin] - ro[fin]) <= tol).all()


FAR_POISON = [
    # cap, len, Np, poisoned slot (own if None: the prefix's), rows a K/V head: undivided, divided, and both behind a prefix
    (500, 490, 0, 5, 2),
    (4096, 4000, 0, 5, 2),
    (4096, 4000, 0, 5, 40),
    (300, 300, 700, 5, 2),
    (300, 300, 700, None, 2),
    (2000, 1999, 400, 5, 150),
    (2000, 1999, 400, None, 150),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("cap,n,Np,at,Hq", FAR_POISON)
def test_poison_far_below_the_largest_score_is_not_lost(fmt, D, cap, n, Np, at, Hq):
    """A visible V row of NaN whose score lies 256 below others, more than a
    weight in fp32 can show: 0 times NaN is NaN however the keys are divided."""
    dev = _gpu()
    kc, vc, ks, vs = new_cache(1, 1, cap, D, fmt, dev)
    heavy = torch.zeros(1, 1, n, D)
    g = torch.Generator().manual_seed(3)
    heavy[..., 1:] = 0.1 * torch.randn(1, 1, n, D - 1, generator=g)
    pk, pv = ((rows(1, 1, Np, D, 5, sigma=0.1)[0].contiguous(), rows(1, 1, Np, D, 6)[0].contiguous()) if Np else (None, None))
    if Np and at is not None:
        pk[:, 50:, 0] = 16 * D ** 0.5          # the prefix outweighs the sequence's own keys
    else:
        heavy[:, :, n - 100:, 0] = 16 * D ** 0.5
    cache.cache_write(heavy.to(torch.bfloat16).to(dev), rows(1, 1, n, D, 2), kc, vc, ints(0), k_scale=ks, v_scale=vs)
    q = rows(1, Hq, 1, D, 3, sigma=0.1).clone()
    q[..., 0] = 16
    clean = cache.decode_cache(q, kc, vc, ints(n), ks, vs, pk, pv)
    assert torch.isfinite(clean[0]).all()
    if at is None:
        pv[0, 5, 7] = float("nan")
    elif fmt == "bf16":
        vc[0, 0, at, 7] = float("nan")
    else:
        vs[0, 0, at] = float("nan")
    o, lse = cache.decode_cache(q, kc, vc, ints(n), ks, vs, pk, pv)
    assert A.device_status(dev) == A.FA_OK
    assert torch.equal(lse, clean[1])
    bad = torch.zeros(D, dtype=torch.bool, device=dev)
    if at is None or fmt == "bf16":
        bad[7] = True
    else:
        bad[:] = True
    assert torch.isnan(o[..., bad]).all() and torch.equal(o[..., ~bad], clean[0][..., ~bad])


def test_many_rows_over_a_long_cache():
    """131072 query rows of 16384 a K/V head, caches of 2^20 slots: far more row
    blocks than CTAs fit at once, each over all of its sequence."""
    dev = _gpu()
    B, Hq, Nq, cap, D = 8, 128, 128, 1 << 20, 64
    lens = [700, 130, 0, 1, 64, 5, 128, 999]
    kc, vc, ks, vs = filled(B, 1, cap, D, "e4m3", lens, dev)
    q = rows(B, Hq, Nq, D, 3)
    o, lse = cache.decode_cache(q, kc, vc, ints(*lens), ks, vs)
    assert A.device_status(dev) == A.FA_OK, f"sites {A.timeout_sites():#x}"
    near = [t[:, :, :1000] for t in (kc, vc, ks, vs)]
    check_decode(q[:, 5::32], *near, ints(*lens), (o[:, 5::32], lse[:, 5::32]))


def test_many_rows_behind_a_long_prefix():
    """131072 query rows over a prefix of 2^21 + 100 keys.  A part adds up to
    16385 key tiles one after another, so sums in fp32 are off by up to 16385
    2^-24 of their magnitudes (twice: numerator and sum)."""
    dev = _gpu()
    B, Hq, Nq, D, Np = 8, 128, 128, 64, (1 << 21) + 100
    kc, vc, ks, vs = filled(B, 1, 4, D, "int8", [4] * B, dev)
    q = rows(B, Hq, Nq, D, 3)
    pk, pv = rows(1, 1, Np, D, 5)[0].contiguous(), rows(1, 1, Np, D, 6)[0].contiguous()
    o, lse = cache.decode_cache(q, kc, vc, ints(*[4] * B), ks, vs, pk, pv)
    assert A.device_status(dev) == A.FA_OK, f"sites {A.timeout_sites():#x}"
    k, v, fk, fv = values(kc, ks), values(vc, vs), np64(pk)[0], np64(pv)[0]
    sums = 16385 * 2.0 ** -24
    for b, h, i in ((0, 0, 0), (3, 64, 126), (7, 127, 127)):
        own = max(4 - Nq + i + 1, 0)
        ro, rl, wt, size = so.decode_rows(np64(q[b, h, i]), np.concatenate([fk, k[b, 0, :own]]),
                                          np.concatenate([fv, v[b, 0, :own]]), D ** -0.5, np.ones(Np + own, dtype=bool))
        ds = (D + 16) * 2.0 ** -23 * size
        tol = (BF * 1.01 + 2 * ds + 2 * sums + 2.0 ** -18) * wt + BF * 1.01 * np.abs(ro)
        assert (np.abs(np64(o[b, h, i]) - ro) <= tol).all()
        assert abs(float(lse[b, h, i]) - rl) <= ds + sums + 2.0 ** -18 + 2.0 ** -22 * abs(rl)


PREFIX_DIVIDED = [
    # B, Hq, Hkv, Nq, cap, D, Np, lens, causal: caches whose heads several CTAs share, behind a prefix, 5 to 100 rows a head
    (2, 16, 1, 4, 700, 128, 200, [700, 3], True),               # two row blocks; one row tile of the prefix, full
    (3, 33, 1, 1, 1032, 64, 300, [1031, 0, 513], True),         # a row block of one row
    (2, 9, 1, 1, 600, 64, 130, [600, 599], False),
    (5, 32, 2, 2, 900, 128, 500, [900, 1, 64, 65, 899], True),  # two row tiles share the prefix's keys
    (2, 50, 1, 2, 520, 128, 129, [519, 2], False),              # four row blocks
    (1, 12, 4, 3, 3000, 64, 1000, [2999], True),
    (40, 10, 2, 1, 516, 64, 64, [(13 * b) % 517 for b in range(40)], False),
    (16, 64, 2, 1, 640, 128, 300, [40 * b for b in range(16)], True),   # as many rows as the join gives a warp each
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,cap,D,Np,lens,causal", PREFIX_DIVIDED)
def test_divided_caches_behind_a_prefix(fmt, B, Hq, Hkv, Nq, cap, D, Np, lens, causal):
    dev = _gpu()
    kc, vc, ks, vs = filled(B, Hkv, cap, D, fmt, lens, dev, seed=51)
    q = rows(B, Hq, Nq, D, 52)
    pk, pv = rows(1, Hkv, Np, D, 53)[0].contiguous(), rows(1, Hkv, Np, D, 54)[0].contiguous()
    got = cache.decode_cache(q, kc, vc, ints(*lens), ks, vs, pk, pv, causal=causal)
    assert A.device_status(dev) == A.FA_OK, f"sites {A.timeout_sites():#x}"
    check_decode(q, kc, vc, ks, vs, ints(*lens), got, causal, pk=pk, pv=pv)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_reading_no_slots(fmt):
    """The history of sequences that have none yet, as writing no rows."""
    dev = _gpu()
    kc, vc, ks, vs = filled(2, 3, 64, 64, fmt, [64, 5], dev)
    k, v = cache.cache_read(kc, vc, 0, lens=ints(0, 0), k_scale=ks, v_scale=vs)
    assert k.shape == v.shape == (2, 3, 0, 64) and k.dtype == torch.bfloat16 and k.is_cuda
    with pytest.raises((TypeError, ValueError, RuntimeError)):
        cache.cache_read(kc, vc, -1, k_scale=ks, v_scale=vs)
    with pytest.raises((TypeError, ValueError)):
        cache.cache_read(kc, vc, 0, lens=[0, 0], k_scale=ks, v_scale=vs)
