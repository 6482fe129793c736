"""GPU parity of qk_norm_rope and its backward against the fp64 definitions.

Tolerances, from the arithmetic: a bf16 result is off by half a step (2^-8 of
its value); before that, fp32 sums of D squares in 8 + log2(D / 8) steps, a
reciprocal root and three products leave at most 32 units of 2^-24 of the
magnitudes that meet, and the angles' turns 2^-22.  A weight's gradient adds at
most `depth` terms in a row in any order of the partial sums, so it is off by
(depth + 32) 2^-24 of the sum of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from tiled_attention_16_b200 import attention as A
from tiled_attention_16_b200 import rope

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.finfo(torch.bfloat16).eps / 2


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def np64(t):
    return t.detach().double().cpu().numpy()


def make(B, Hq, Hkv, N, D, rot, layout="packed", wdtype=torch.float32, seed=0, first=0):
    dev = _gpu()
    g = torch.Generator().manual_seed(seed)
    if layout == "packed":
        qkv = torch.randn(B, N, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).to(dev)
        q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    elif layout == "head_major":
        q = torch.randn(B, Hq, N, D, generator=g).to(torch.bfloat16).to(dev)
        k = torch.randn(B, Hkv, N, D, generator=g).to(torch.bfloat16).to(dev)
    else:   # padded rows and an offset of 8 elements: 16-byte alignment only
        buf = torch.randn(B * N * (Hq + Hkv) * (D + 24) + 8, generator=g).to(torch.bfloat16).to(dev)
        both = buf[8:].view(B, N, Hq + Hkv, D + 24)[..., 16:16 + D]
        q, k = both[:, :, :Hq].transpose(1, 2), both[:, :, Hq:].transpose(1, 2)
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(wdtype).to(dev) for _ in range(2))
    inv = (1.0 / 10000.0 ** (torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(dev)
    pos = (torch.arange(N, dtype=torch.int32)[None] + first * torch.arange(1, B + 1, dtype=torch.int32)[:, None])
    dq = torch.randn(B, Hq, N, D, generator=g).to(torch.bfloat16).to(dev)
    dk = torch.randn(B, Hkv, N, D, generator=g).to(torch.bfloat16).to(dev)
    return q, k, qw, kw, inv, pos.contiguous().to(dev), dq, dk


def check_forward(q, k, qw, kw, inv, pos, out, eps, inter):
    for x, w, y in ((q, qw, out[0]), (k, kw, out[1])):
        ref, u = so.norm_rope(np64(x), np64(w), np64(inv), pos.cpu().numpy(), eps, inter)
        top = np.abs(u).max(-1, keepdims=True)
        assert (np.abs(np64(y) - ref) <= BF * np.abs(ref) * (1 + BF) + 2 * (32 * U + 2.0 ** -22) * top).all()


def check_backward(q, k, qw, kw, inv, pos, dq, dk, got, eps, inter, depth):
    for x, w, dy, dx, dw in ((q, qw, dq, got[0], got[2]), (k, kw, dk, got[1], got[3])):
        rdx, rdw, sdx, sdw = so.norm_rope_backward(np64(dy), np64(x), np64(w), np64(inv), pos.cpu().numpy(), eps, inter)
        slack = 32 * U + 2.0 ** -22
        assert (np.abs(np64(dx) - rdx) <= BF * np.abs(rdx) * (1 + BF) + slack * sdx + 2.0 ** -133).all()
        assert (np.abs(np64(dw) - rdw) <= ((depth + 32) * U + 2.0 ** -22) * sdw + 1e-37).all()


CASES = [
    # B, Hq, Hkv, N, D, rot, interleaved, layout, weights, first position
    (1, 1, 1, 1, 128, 128, False, "packed", torch.float32, 0),
    (2, 4, 2, 5, 128, 128, True, "packed", torch.bfloat16, 7),
    (3, 12, 4, 37, 64, 32, True, "packed", torch.bfloat16, 100),
    (2, 5, 3, 33, 128, 48, False, "padded", torch.float32, 1 << 20),
    (1, 7, 1, 130, 64, 64, False, "head_major", torch.float32, 0),
    (5, 64, 8, 1, 128, 128, False, "packed", torch.bfloat16, 400000000),
    (2, 3, 5, 19, 64, 8, False, "padded", torch.float32, 3),
    (1, 2, 2, 300, 128, 0, False, "packed", torch.float32, 0),
    (1, 9, 9, 257, 128, 24, True, "packed", torch.bfloat16, 5),
]


@pytest.mark.parametrize("B,Hq,Hkv,N,D,rot,inter,layout,wt,first", CASES)
def test_forward_and_backward(B, Hq, Hkv, N, D, rot, inter, layout, wt, first):
    q, k, qw, kw, inv, pos, dq, dk = make(B, Hq, Hkv, N, D, rot, layout, wt, seed=N + D, first=first)
    eps = 1e-5
    kwargs = dict(positions=pos, eps=eps, interleaved=inter)
    f = inv if rot else None
    out = rope.qk_norm_rope(q, k, qw, kw, f, **kwargs)
    assert out[0].is_contiguous() and out[1].is_contiguous()
    check_forward(q, k, qw, kw, inv, pos, out, eps, inter)
    got = rope.qk_norm_rope_bwd(dq, dk, q, k, qw, kw, f, **kwargs)
    check_backward(q, k, qw, kw, inv, pos, dq, dk, got, eps, inter, depth=B * N * max(Hq, Hkv))


def test_many_tokens_walk_several_items():
    """More items than CTAs in the backward: every CTA walks several."""
    q, k, qw, kw, inv, pos, dq, dk = make(2, 3, 1, 30000, 64, 64, seed=3)
    got = rope.qk_norm_rope_bwd(dq, dk, q, k, qw, kw, inv, positions=pos, eps=1e-6)
    check_backward(q, k, qw, kw, inv, pos, dq, dk, got, 1e-6, False, depth=1024)
    again = rope.qk_norm_rope_bwd(dq, dk, q, k, qw, kw, inv, positions=pos, eps=1e-6)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_default_positions_and_outputs():
    q, k, qw, kw, inv, pos, dq, dk = make(2, 4, 2, 50, 128, 128, seed=8)
    ref = rope.qk_norm_rope(q, k, qw, kw, inv, positions=pos)
    oq, ok = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    got = rope.qk_norm_rope(q, k, qw, kw, inv, out_q=oq, out_k=ok)
    assert got[0] is oq and torch.equal(oq, ref[0]) and torch.equal(ok, ref[1])
    # gradients into views of one packed buffer; its other rows stay
    packed = torch.full((2, 50, 4 + 2 * 2, 128), 3.0, device=q.device, dtype=torch.bfloat16)
    want = rope.qk_norm_rope_bwd(dq, dk, q, k, qw, kw, inv)
    res = rope.qk_norm_rope_bwd(dq, dk, q, k, qw, kw, inv, dq=packed[:, :, :4].transpose(1, 2),
                                dk=packed[:, :, 4:6].transpose(1, 2))
    assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1])
    assert (packed[:, :, 6:] == 3.0).all()
    assert torch.equal(res[2], want[2]) and torch.equal(res[3], want[3])


def test_negative_and_extreme_positions():
    q, k, qw, kw, inv, _, _, _ = make(1, 2, 1, 4, 128, 128, seed=5)
    pos = torch.tensor([[-1, -(2 ** 31), 2 ** 31 - 1, 12345]], dtype=torch.int32, device=q.device)
    out = rope.qk_norm_rope(q, k, qw, kw, inv, positions=pos, eps=1e-6)
    for x, w, y in ((q, qw, out[0]), (k, kw, out[1])):
        ref, u = so.norm_rope(np64(x), np64(w), np64(inv), pos.cpu().numpy(), 1e-6, False)
        # 2^31 / (2 pi) turns: the product and the reduction in fp64 leave 2^-53 * 2^28.4 turns, 3e-7 rad
        assert (np.abs(np64(y) - ref) <= 1.01 * BF * np.abs(ref) + 4e-6 * np.abs(u).max(-1, keepdims=True)).all()


def test_zero_rows_and_values_that_poison_one_row():
    q, k, qw, kw, inv, pos, dq, dk = make(1, 3, 2, 6, 64, 64, seed=6, layout="head_major")
    q[0, 1, 2] = 0
    q[0, 2, 3, 5] = float("nan")
    k[0, 0, 4, 1] = float("inf")
    oq, ok = rope.qk_norm_rope(q, k, qw, kw, inv, positions=pos)
    assert (oq[0, 1, 2] == 0).all()
    assert torch.isnan(oq[0, 2, 3]).all() and torch.isfinite(oq[0, :2]).all() and torch.isfinite(oq[0, 2, :3]).all()
    assert torch.isnan(ok[0, 0, 4]).any() and torch.isfinite(ok[0, 1]).all() and torch.isfinite(ok[0, 0, :4]).all()


def test_gradient_against_differences():
    """dL for L = <y, dy> along random directions, by central differences of
    the fp64 definition."""
    q, k, qw, kw, inv, pos, dq, dk = make(1, 2, 1, 3, 64, 64, seed=12)
    got = rope.qk_norm_rope_bwd(dq, dk, q, k, qw, kw, inv, positions=pos, eps=1e-5)
    rng = np.random.default_rng(0)
    p = pos.cpu().numpy()
    for x, w, dy, dx, dw in ((q, qw, dq, got[0], got[2]), (k, kw, dk, got[1], got[3])):
        x, w, dy = np64(x), np64(w), np64(dy)
        f = lambda a, c: (so.norm_rope(a, c, np64(inv), p, 1e-5, False)[0] * dy).sum()  # noqa: E731
        ex, ew, h = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-5
        num = (f(x + h * ex, w) - f(x - h * ex, w)) / (2 * h)
        assert abs((np64(dx) * ex).sum() - num) <= BF * np.abs(np64(dx) * ex).sum() + 1e-5
        num = (f(x, w + h * ew) - f(x, w - h * ew)) / (2 * h)
        assert abs((np64(dw) * ew).sum() - num) <= 1e-5 * (1 + np.abs(np64(dw) * ew).sum())


def test_offsets_past_32_bits():
    """More than 2^31 elements: sampled rows against the definition."""
    dev = _gpu()
    N, Hq, Hkv, D = 150000, 112, 8, 128
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.empty(1, N, Hq + Hkv, D, device=dev, dtype=torch.bfloat16)
    for i in range(0, N, 10000):
        x[:, i:i + 10000] = torch.randn(1, 10000, Hq + Hkv, D, device=dev, generator=g, dtype=torch.float32)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:].transpose(1, 2)
    assert q.numel() > 1 << 31
    w = torch.ones(D, device=dev)
    inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(dev)
    oq, ok = rope.qk_norm_rope(q, k, w, w, inv)
    dq, dk, dqw, dkw = rope.qk_norm_rope_bwd(oq, ok, q, k, w, w, inv)
    for t, y, d, heads in ((q, oq, dq, (0, 57, Hq - 1)), (k, ok, dk, (0, Hkv - 1))):
        for h in heads:
            for n in (0, 77777, N - 1):
                pos = np.array([[n]])
                ref, u = so.norm_rope(np64(t[:, h:h + 1, n:n + 1]), np.ones(D), np64(inv), pos, 1e-6, False)
                assert (np.abs(np64(y[0, h, n]) - ref[0, 0, 0]) <= BF * np.abs(ref[0, 0, 0]) * (1 + BF) + 1e-5).all()
                rdx, _, sdx, _ = so.norm_rope_backward(np64(y[:, h:h + 1, n:n + 1]), np64(t[:, h:h + 1, n:n + 1]),
                                                       np.ones(D), np64(inv), pos, 1e-6, False)
                assert (np.abs(np64(d[0, h, n]) - rdx[0, 0, 0]) <= BF * np.abs(rdx[0, 0, 0]) * (1 + BF) + 1e-5 * sdx[0, 0, 0]).all()
    # dy = y of the same rows, so g x r = x^2 r^2 (1 +- 2^-8): the sums are the rows' count, about
    for dw, H in ((dqw, Hq), (dkw, Hkv)):
        assert (np64(dw) / (N * H)).min() > 0.98 and (np64(dw) / (N * H)).max() < 1.02
    del x, q, k, oq, ok, dq, dk
    torch.cuda.empty_cache()


def test_refusals_on_the_gpu():
    q, k, qw, kw, inv, pos, dq, dk = make(1, 2, 1, 4, 64, 64, seed=2)
    ok = dict(positions=pos)
    for args, kwargs in (((q.float(), k, qw, kw, inv), ok), ((q[..., ::2], k[..., ::2], qw[:32], kw[:32], inv), ok),
                         ((q, k, qw.half(), kw, inv), ok), ((q, k, qw, kw.bfloat16(), inv), ok),
                         ((q, k, qw, kw, inv.double()), ok), ((q, k, qw, kw, inv), dict(positions=pos.long())),
                         ((q, k, qw, kw, inv), dict(positions=pos[:, :2])), ((q, k, qw, kw, inv), dict(eps=0.0)),
                         ((q, k, qw, kw, inv[:3]), ok), ((q, k[:, :, :3], qw, kw, inv), ok),
                         ((q, k, qw, kw.cpu(), inv), ok), ((q, k, qw, kw, inv), dict(out_q=dq[:, :, :, :32]))):
        with pytest.raises((TypeError, ValueError, A.FAError)):
            rope.qk_norm_rope(*args, **kwargs)
    wide = torch.empty(1, 1, 4, 64, device=q.device, dtype=torch.bfloat16)
    for bad in (dict(dq=wide.expand(1, 2, 4, 64)), dict(workspace=torch.empty(8, device=q.device)),
                dict(workspace=torch.empty(1, device=q.device).expand(1 << 30)), dict(dk=dk.float())):
        with pytest.raises((TypeError, ValueError, A.FAError)):
            rope.qk_norm_rope_bwd(dq, dk, q, k, qw, kw, inv, **bad)
    assert A.device_status(q.device) == A.FA_OK


def test_refusals_of_what_is_no_tensor():
    q, k, qw, kw, inv, pos, dq, dk = make(1, 2, 1, 4, 64, 64, seed=2)
    for args in ((None, k, qw, kw, inv), (q, None, qw, kw, inv), (q, k, None, kw, inv), (q, k, qw, None, inv),
                 (q, k, qw, kw, [1.0]), (q, k, qw, kw, inv, [0, 1, 2, 3])):
        with pytest.raises((TypeError, ValueError)):
            rope.qk_norm_rope(*args)
    for args, more in (((None, dk), {}), ((dq, None), {}), ((dq, dk), dict(workspace=7)), ((dq, dk), dict(dq=3))):
        with pytest.raises((TypeError, ValueError)):
            rope.qk_norm_rope_bwd(*args, q, k, qw, kw, inv, **more)
    assert A.device_status(q.device) == A.FA_OK


def test_broadcast_inputs():
    """Views whose rows repeat (stride 0) are read like any other."""
    q, k, qw, kw, inv, pos, dq, dk = make(2, 4, 2, 9, 128, 64, seed=4)
    qe, ke = q[:, :1].expand(-1, 4, -1, -1), k[:1].expand(2, -1, -1, -1)
    a = rope.qk_norm_rope(qe, ke, qw, kw, inv, positions=pos)
    b = rope.qk_norm_rope(qe.contiguous(), ke.contiguous(), qw, kw, inv, positions=pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = rope.qk_norm_rope_bwd(dq, dk, qe, ke, qw, kw, inv, positions=pos)
    gb = rope.qk_norm_rope_bwd(dq, dk, qe.contiguous(), ke.contiguous(), qw, kw, inv, positions=pos)
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))


def test_graph_capture_and_other_stream():
    q, k, qw, kw, inv, pos, dq, dk = make(2, 4, 2, 65, 128, 128, seed=14)
    want = rope.qk_norm_rope(q, k, qw, kw, inv, positions=pos) + rope.qk_norm_rope_bwd(
        dq, dk, q, k, qw, kw, inv, positions=pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = rope.qk_norm_rope(q, k, qw, kw, inv, positions=pos) + rope.qk_norm_rope_bwd(
            dq, dk, q, k, qw, kw, inv, positions=pos)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = rope.qk_norm_rope(q, k, qw, kw, inv, positions=pos) + rope.qk_norm_rope_bwd(
            dq, dk, q, k, qw, kw, inv, positions=pos)
    pos += 11
    g.replay()
    torch.cuda.synchronize()
    want = rope.qk_norm_rope(q, k, qw, kw, inv, positions=pos) + rope.qk_norm_rope_bwd(
        dq, dk, q, k, qw, kw, inv, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(want, res))


def test_training_step_with_attention():
    """qk_norm_rope -> fwd -> bwd -> qk_norm_rope_bwd against the composed fp64
    definitions, at the attention gradients' relative tolerance."""
    import oracle
    B, Hq, Hkv, N, D = 1, 4, 2, 200, 128
    q, k, qw, kw, inv, pos, _, _ = make(B, Hq, Hkv, N, D, D, seed=21)
    g = torch.Generator().manual_seed(22)
    v = torch.randn(B, Hkv, N, D, generator=g).to(torch.bfloat16).to(q.device)
    do = torch.randn(B, Hq, N, D, generator=g).to(torch.bfloat16).to(q.device)
    rq, rk = rope.qk_norm_rope(q, k, qw, kw, inv, positions=pos)
    o, lse = A.fwd(rq, rk, v, causal=True)
    drq, drk, dv = A.bwd(rq, rk, v, o, do, lse, causal=True)
    got = rope.qk_norm_rope_bwd(drq, drk, q, k, qw, kw, inv, positions=pos)
    assert A.device_status(q.device) == A.FA_OK
    p = pos.cpu().numpy()
    yq, yk = (so.norm_rope(np64(x), np64(w), np64(inv), p, 1e-6, False)[0] for x, w in ((q, qw), (k, kw)))
    gq, gk, gv = oracle.attention_backward(torch.from_numpy(yq), torch.from_numpy(yk), v.cpu(), do.cpu(), D ** -0.5, True)
    rdq, rdqw, _, _ = so.norm_rope_backward(gq, np64(q), np64(qw), np64(inv), p, 1e-6, False)
    rdk, rdkw, _, _ = so.norm_rope_backward(gk, np64(k), np64(kw), np64(inv), p, 1e-6, False)
    for a, b in ((got[0], rdq), (got[1], rdk), (got[2], rdqw), (got[3], rdkw), (dv, gv)):
        assert np.linalg.norm(np64(a) - b) <= 2e-2 * np.linalg.norm(b)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("top", [1.0, 1e3, 3e5, 1e17, 3e38])
def test_angles_of_any_size(top, inter):
    """Frequencies far from 1 at the largest positions, against angles reduced
    in integers: within 2^-31 + 2^-106 |angle| of a turn, then fp32."""
    dev = _gpu()
    D, rot = 64, 64
    q, k, qw, kw, _, _, dq, dk = make(2, 3, 2, 8, D, rot, seed=21)
    inv = torch.from_numpy(np.geomspace(1e-6, top, rot // 2).astype(np.float32)).to(dev)
    pos = torch.tensor([[0, 1, -1, 77, 1000001, -123456789, 2 ** 31 - 1, -(2 ** 31)],
                        [3, 2 ** 30, 5, 2 ** 31 - 2, 2, 65537, 12345, 4096]], dtype=torch.int32, device=dev)
    eps = 1e-6
    got = rope.qk_norm_rope(q, k, qw, kw, inv, positions=pos, eps=eps, interleaved=inter)
    grads = rope.qk_norm_rope_bwd(dq, dk, q, k, qw, kw, inv, positions=pos, eps=eps, interleaved=inter)
    far = 2 * np.pi * (2.0 ** -31 + 2.0 ** -106 * float(inv.max()) * 2.0 ** 31)
    assert far < 2.0 ** -10 or top > 1e30
    slack = 32 * U + 2.0 ** -22 + min(far, 2.0)
    for x, w, dy, y, dx, dw in ((q, qw, dq, got[0], grads[0], grads[2]), (k, kw, dk, got[1], grads[1], grads[3])):
        args = (np64(x), np64(w), np64(inv), pos.cpu().numpy(), eps, inter, so.reduced_angles)
        ref, u = so.norm_rope(*args)
        size = np.abs(u).max(-1, keepdims=True)
        assert (np.abs(np64(y) - ref) <= BF * np.abs(ref) * (1 + BF) + 2 * slack * size).all()
        rdx, rdw, sdx, sdw = so.norm_rope_backward(np64(dy), *args)
        assert (np.abs(np64(dx) - rdx) <= BF * np.abs(rdx) * (1 + BF) + slack * sdx + 2.0 ** -133).all()
        assert (np.abs(np64(dw) - rdw) <= ((2 * 8 * 3 + 32) * U + slack) * sdw).all()
