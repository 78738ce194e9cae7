"""The per-head norms of q and k with the position rotation, their gradients and
the 8-bit checkpoint, against the formulas in fp64.

Tolerances (relative L2): fp32 results TOL_F32; results stored in bf16 also get
half a bf16 step, 2^-8 of each value. Codes and scales are compared exactly.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from tests.parity import TOL_BF16, TOL_F32, assert_close, np64

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def tol(dtype):
    return TOL_F32 + (torch.finfo(dtype).eps / 2 if dtype == BF else 0.0)


def inv_freq(rot, base=10000.0, stretch=1.0):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / stretch


def plain(x, w, how, scale=1.0):
    """The definition, fp64: x [T,H,d] -> y."""
    x = x.double()
    ss = (x * x).sum(-1, keepdim=True)
    eps = how.get("eps", 1e-6)
    if how["norm"] == "l2":
        x = x / torch.sqrt(ss + eps)
    elif how["norm"] == "rms":
        x = x / torch.sqrt(ss / x.shape[-1] + eps)
    if w is not None:
        x = x * (w.double() + how.get("weight_offset", 0.0))
    f = how.get("inv_freq")
    if f is not None:
        r = 2 * f.numel()
        a = how["positions"].double()[:, None, None] * f
        c, s = a.cos() * how.get("rope_scale", 1.0), a.sin() * how.get("rope_scale", 1.0)
        if how.get("interleaved"):
            u, v = x[..., 0:r:2], x[..., 1:r:2]
            turned = torch.stack([u * c - v * s, v * c + u * s], -1).flatten(-2)
        else:
            u, v = x[..., :r // 2], x[..., r // 2:r]
            turned = torch.cat([u * c - v * s, v * c + u * s], -1)
        x = torch.cat([turned, x[..., r:]], -1)
    return x * scale


def plain_pack(x):
    """Codes as values, and scales, by search: the e4m3 value nearest to x / 2^e, ties to the even code."""
    T, H, d = x.shape
    table = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()     # 0 .. 448
    blocks = torch.nn.functional.pad(x.double(), (0, -d % 32)).unflatten(-1, (-1, 32))
    fine = torch.isfinite(blocks)
    top = torch.where(fine, blocks.abs(), 0.0).amax(-1)
    e = torch.full(top.shape, -127.0, dtype=torch.float64)
    for i in range(-126, 122):
        e = torch.where(top > 448.0 * 2.0 ** (i - 1), float(i), e)
    y = torch.where(fine, blocks, 0.0) / torch.exp2(e)[..., None]
    hi = torch.searchsorted(table, y.abs().contiguous()).clamp_max(126)
    lo = (hi - 1).clamp_min(0)
    dl, dh = y.abs() - table[lo], table[hi] - y.abs()
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    v = torch.where(fine, torch.copysign(table[pick], y), float("nan"))
    return v.flatten(-2)[..., :d], (e + 127).to(torch.uint8)


def value(p):
    """What 8-bit rows stand for, fp64."""
    c, s = p.codes.cpu().double(), p.scales.cpu().double()
    return c * torch.exp2(s - 127).repeat_interleave(32, -1)[..., :c.shape[-1]]


def make(T, Hq, Hk, d, dtype, rot=0, norm="l2", weights=False, interleaved=False, seed=0, far=False,
         **more):
    gen = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(T, h, d, generator=gen).to(dtype) for h in (Hq, Hk))
    how = dict(norm=norm, interleaved=interleaved, **more)
    if rot:
        how["inv_freq"] = inv_freq(rot, stretch=4.0 if far else 1.0)
        how["positions"] = torch.randint(0, (1 << 30) if far else 8192, (T,), generator=gen).to(torch.int32)
    w = [(1 + 0.3 * torch.randn(d, generator=gen)).to(dtype) if weights else None for _ in "qk"]
    return q, k, w, how


def dev(how, w):
    h = {a: b.cuda() if torch.is_tensor(b) else b for a, b in how.items()}
    return dict(h, w_q=None if w[0] is None else w[0].cuda(), w_k=None if w[1] is None else w[1].cuda())


CASES = [
    # T, Hq, Hk, d, dtype, rot, norm, weights, interleaved, more
    (1, 1, 1, 128, BF, 0, "l2", False, False, {}),
    (5, 16, 16, 128, BF, 128, "l2", False, False, dict(q_scale=128 ** -0.5)),
    (7, 8, 2, 128, BF, 64, "rms", True, False, dict(rope_scale=1.3)),
    (9, 3, 5, 128, F, 128, "rms", True, True, dict(weight_offset=1.0)),
    (33, 33, 1, 96, BF, 48, "l2", True, True, {}),
    (33, 17, 4, 96, F, 40, "none", False, False, {}),        # halves that meet inside a lane
    (4, 2, 3, 80, BF, 80, "rms", False, False, {}),
    (6, 5, 5, 132, BF, 66, "l2", True, False, {}),
    (3, 4, 2, 256, BF, 256, "rms", True, False, {}),
    (3, 4, 2, 200, F, 96, "l2", False, False, {}),
    (2, 3, 1, 36, BF, 36, "none", True, True, {}),
    (3, 2, 2, 33, BF, 2, "rms", True, False, {}),
    (2, 2, 7, 1, F, 0, "l2", False, False, {}),
    (2, 1, 2, 7, F, 6, "rms", False, True, {}),
    (1200, 4, 1, 64, BF, 32, "l2", True, False, {}),
]


def setup(case, **more):
    T, Hq, Hk, d, dtype, rot, norm, weights, inter, extra = CASES[case]
    return make(T, Hq, Hk, d, dtype, rot, norm, weights, inter, seed=case, far=case % 2 == 1,
                **{**extra, **more})


@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward(case):
    import gated_delta_rule_112_b200 as gdn
    q, k, w, how = setup(case)
    yq, yk = gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), **dev(how, w))
    rh = {a: b for a, b in how.items() if a != "q_scale"}
    assert_close("q", np64(yq), plain(q, w[0], rh, how.get("q_scale", 1.0)).numpy(), tol(q.dtype))
    assert_close("k", np64(yk), plain(k, w[1], rh).numpy(), tol(q.dtype))


def grads_of(x, w, how, scale, dy):
    x = x.double().requires_grad_()
    w = None if w is None else w.double().requires_grad_()
    plain(x, w, how, scale).backward(dy.double())
    return x.grad.numpy(), None if w is None else w.grad.numpy()


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("grad", [F, None])
def test_backward(case, grad):
    """Against the formula's gradients in fp64 (by automatic differentiation)."""
    import gated_delta_rule_112_b200 as gdn
    q, k, w, how = setup(case)
    gt = grad or q.dtype
    gen = torch.Generator().manual_seed(100 + case)
    dy = [torch.randn(x.shape, generator=gen).to(gt) for x in (q, k)]
    out = gdn.qk_norm_rope_bwd(dy[0].cuda(), dy[1].cuda(), q.cuda(), k.cuda(), **dev(how, w))
    rh = {a: b for a, b in how.items() if a != "q_scale"}
    for i, (x, n) in enumerate(((q, "q"), (k, "k"))):
        dx, dw = grads_of(x, w[i], rh, how.get("q_scale", 1.0) if i == 0 else 1.0, dy[i])
        # a row's gradient can cancel (d = 1: to nothing), so against the terms it is made of
        if q.shape[-1] > 1:
            assert_close("d" + n, np64(out["d" + n]), dx, tol(q.dtype))
        if dw is None:
            assert out["dw_" + n] is None
        else:
            assert_close("dw_" + n, np64(out["dw_" + n]), dw, TOL_F32)


def test_backward_against_differences():
    """Central differences of the GPU forward itself, fp32, step h = 2^-6: the truncation is
    h^2 f''' / 6 ~ 4e-5 and the rounding 2^-24 / h ~ 4e-6 of the loss's scale, so 1e-3 of the gradient's."""
    import gated_delta_rule_112_b200 as gdn
    q, k, w, how = make(2, 2, 1, 8, F, 6, "rms", True, False, seed=50, eps=1e-2)
    gen = torch.Generator().manual_seed(51)
    dy = [torch.randn(x.shape, generator=gen) for x in (q, k)]
    out = gdn.qk_norm_rope_bwd(dy[0].cuda(), dy[1].cuda(), q.cuda(), k.cuda(), **dev(how, w))

    def loss(q, k, w):
        y = gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), **dev(how, w))
        return sum(float((a.double().cpu() * b.double()).sum()) for a, b in zip(y, dy))

    h = 2.0 ** -6
    for name, x, put in (("dq", q, lambda z: (z, k, w)), ("dk", k, lambda z: (q, z, w)),
                         ("dw_q", w[0], lambda z: (q, k, [z, w[1]])),
                         ("dw_k", w[1], lambda z: (q, k, [w[0], z]))):
        num = torch.zeros(x.shape, dtype=torch.float64)
        for i in range(x.numel()):
            a, b = x.clone(), x.clone()
            a.view(-1)[i] += h
            b.view(-1)[i] -= h
            num.view(-1)[i] = (loss(*put(a)) - loss(*put(b))) / (2 * h)
        assert_close(name, np64(out[name]), num.numpy(), 1e-3)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_codes_are_exact(case):
    import gated_delta_rule_112_b200 as gdn
    q, k, w, how = setup(case)
    q = q * torch.exp2(torch.arange(q.shape[0]) % 60 - 30.0)[:, None, None].to(q.dtype)
    yq, yk, q8, k8 = gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), pack=True, **dev(how, w))
    for x, p in ((q, q8), (k, k8)):
        codes, scales = plain_pack(x)
        assert torch.equal(p.scales.cpu(), scales)
        assert torch.equal(p.codes.cpu().double(), codes)
    zq, zk = gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), **dev(how, w))     # the codes change no output
    assert torch.equal(yq, zq) and torch.equal(yk, zk)


def test_codes_at_the_ends():
    """Zeros, infinities and NaN, the smallest and largest values, a block of one kind beside another."""
    import gated_delta_rule_112_b200 as gdn
    for dtype in (BF, F):
        top = torch.finfo(dtype).max
        x = torch.zeros(9, 2, 72, dtype=dtype)
        x[1] = top
        x[2] = 2.0 ** -133                       # below the normal range
        x[3, 0, 5], x[3, 0, 40], x[3, 1, 3] = math.inf, -math.inf, math.nan
        x[3, :, 6:9], x[3, :, 64:] = 3.0, 0.1
        x[4] = torch.linspace(-448, 448, 72).to(dtype)
        x[5] = 448 * 2.0 ** -126 * 0.5
        x[6] = torch.randn(2, 72).to(dtype) * 2.0 ** -128
        x[7] = -math.inf
        x[8, :, ::2] = 464.0                     # halfway: a step above 448
        p = gdn.pack(x.cuda())
        codes, scales = plain_pack(x)
        assert torch.equal(p.scales.cpu(), scales)
        assert torch.equal(torch.nan_to_num(p.codes.cpu().double(), 999.0), torch.nan_to_num(codes, 999.0))
        back = gdn.unpack(p, dtype)
        # exact, but that the largest values' codes stand for 2^128, an infinity in either type
        assert torch.equal(torch.nan_to_num(back.cpu().double(), 999.0),
                           torch.nan_to_num(value(p).to(dtype).double(), 999.0))


@pytest.mark.parametrize("case", range(len(CASES)))
def test_from_the_checkpoint(case):
    """Outputs and gradients from 8-bit rows: the formulas at the values the rows stand for."""
    import gated_delta_rule_112_b200 as gdn
    q, k, w, how = setup(case)
    p = [gdn.pack(x.cuda()) for x in (q, k)]
    x = [value(y) for y in p]
    y = gdn.qk_norm_rope_fwd(*p, dtype=q.dtype, **dev(how, w))
    rh = {a: b for a, b in how.items() if a != "q_scale"}
    scale = [how.get("q_scale", 1.0), 1.0]
    gen = torch.Generator().manual_seed(200 + case)
    dy = [torch.randn(z.shape, generator=gen) for z in (q, k)]
    out = gdn.qk_norm_rope_bwd(dy[0].cuda(), dy[1].cuda(), *p, dtype=q.dtype, **dev(how, w))
    for i, n in enumerate("qk"):
        assert_close(n, np64(y[i]), plain(x[i], w[i], rh, scale[i]).numpy(), tol(q.dtype))
        dx, dw = grads_of(x[i], w[i], rh, scale[i], dy[i])
        if q.shape[-1] > 1:
            assert_close("d" + n, np64(out["d" + n]), dx, tol(q.dtype))
        if dw is not None:
            assert_close("dw_" + n, np64(out["dw_" + n]), dw, TOL_F32)


def test_strided_unaligned_and_in_place():
    import gated_delta_rule_112_b200 as gdn
    for dtype in (BF, F):
        q, k, w, how = make(6, 4, 2, 128, dtype, 64, "rms", True, seed=60)
        rh = dict(how)
        for offset in (0, 1, 4):
            wide = torch.full((6, offset + 4 * 128 + 2 * 160 + 3), 5.0, dtype=dtype, device="cuda")
            a = wide[:, offset:offset + 512].unflatten(1, (4, 128))
            b = wide[:, offset + 512:offset + 832].unflatten(1, (2, 160))[..., :128]   # heads apart
            a.copy_(q)
            b.copy_(k)
            before = wide.clone()
            y = gdn.qk_norm_rope_fwd(a, b, **dev(how, w))
            assert torch.equal(before, wide)
            z = gdn.qk_norm_rope_fwd(a, b, out=(a, b), **dev(how, w))
            assert torch.equal(z[0], y[0]) and torch.equal(z[1], y[1]) and z[0].data_ptr() == a.data_ptr()
            mask = torch.ones_like(wide, dtype=torch.bool)
            mask[:, offset:offset + 512] = False
            mask[:, offset + 512:offset + 832].unflatten(1, (2, 160))[..., :128] = False
            assert torch.equal(wide[mask], before[mask])             # between the heads: untouched
            assert_close("q", np64(y[0]), plain(q, w[0], rh).numpy(), tol(dtype))
            assert_close("k", np64(y[1]), plain(k, w[1], rh).numpy(), tol(dtype))
            a.copy_(q)
            b.copy_(k)
            dy = [torch.randn(x.shape, generator=torch.Generator().manual_seed(3)).to(dtype) for x in (q, k)]
            g1 = gdn.qk_norm_rope_bwd(dy[0].cuda(), dy[1].cuda(), a, b, **dev(how, w))
            g2 = gdn.qk_norm_rope_bwd(dy[0].cuda(), dy[1].cuda(), q.cuda(), k.cuda(), **dev(how, w))
            g3 = gdn.qk_norm_rope_bwd(dy[0].cuda(), dy[1].cuda(), a, b, out=(a, b), **dev(how, w))
            for n in ("dq", "dk"):
                assert_close(n, np64(g1[n]), np64(g2[n]), tol(dtype))
                assert torch.equal(g3[n], g1[n])


def test_heads_outermost():
    """[H, T, d] in memory, as a batch of heads: read, written and taken back through without a copy."""
    import gated_delta_rule_112_b200 as gdn
    q, k, w, how = make(37, 3, 2, 128, BF, 128, "rms", True, seed=61)
    ref = gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), pack=True, **dev(how, w))
    a, b = (x.cuda().transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k))
    y = gdn.qk_norm_rope_fwd(a, b, pack=True, **dev(how, w))
    for i in range(2):
        assert torch.equal(y[i], ref[i])
        assert torch.equal(y[2 + i].codes.view(torch.uint8), ref[2 + i].codes.view(torch.uint8))
    out = tuple(torch.empty(x.shape[1], 37, 128, dtype=BF, device="cuda").transpose(0, 1) for x in (q, k))
    gdn.qk_norm_rope_fwd(a, b, out=out, **dev(how, w))
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    dy = [torch.randn(x.shape, generator=torch.Generator().manual_seed(4)).cuda() for x in (q, k)]
    g = gdn.qk_norm_rope_bwd(*dy, a, b, **dev(how, w))
    want = gdn.qk_norm_rope_bwd(*dy, q.cuda(), k.cuda(), **dev(how, w))
    assert all(torch.equal(g[n], want[n]) for n in want)


def test_far_positions_keep_their_angles():
    """Positions up to 2^31 - 1 and negative ones: fp32 accuracy of the rotation, whatever the turns."""
    import gated_delta_rule_112_b200 as gdn
    pos = torch.tensor([0, 1, -1, 131071, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    f = inv_freq(128)
    q = torch.randn(7, 2, 128, generator=torch.Generator().manual_seed(1))
    how = dict(norm="none", positions=pos, inv_freq=f)
    y, _ = gdn.qk_norm_rope_fwd(q.cuda(), None, norm="none", positions=pos.cuda(), inv_freq=f.cuda())
    ref = plain(q, None, how)
    for t in range(7):       # one turn is known to 2^31 * 2^-53 / 2 pi: nothing beside fp32's 2^-24
        assert_close(f"position {int(pos[t])}", np64(y[t]), ref[t].numpy(), TOL_F32)


def test_offsets_past_32_bits():
    """More than 2^31 elements (and 2^32 bytes): the last token's rows, and the codes of them."""
    import gated_delta_rule_112_b200 as gdn
    T, d = 8_500_000, 256
    x = torch.empty(T, 1, d, dtype=BF, device="cuda")
    last = torch.randn(3, 1, d, generator=torch.Generator().manual_seed(8)).to(BF)
    x[-3:] = last.cuda()
    y, _, p, _ = gdn.qk_norm_rope_fwd(x, None, norm="rms", pack=True)
    assert_close("y", np64(y[-3:]), plain(last, None, dict(norm="rms")).numpy(), tol(BF))
    codes, scales = plain_pack(last)
    assert torch.equal(p.scales[-3:].cpu(), scales) and torch.equal(p.codes[-3:].cpu().double(), codes)
    del y
    out = gdn.qk_norm_rope_bwd(x, None, p, None, norm="rms")
    ref, _ = grads_of(value(gdn.Packed(p.codes[-3:], p.scales[-3:])), None, dict(norm="rms"), 1.0, last)
    assert_close("dx", np64(out["dq"][-3:]), ref, tol(BF))


def test_rows_of_zeros_and_of_infinities():
    import gated_delta_rule_112_b200 as gdn
    q = torch.zeros(3, 2, 128)
    q[1, 0, 3], q[2, 1, 7] = math.inf, math.nan
    y, _ = gdn.qk_norm_rope_fwd(q.cuda(), None, norm="l2")
    assert torch.equal(y[0].cpu(), torch.zeros(2, 128))              # eps keeps a zero row at zero
    assert torch.isnan(y[2, 1]).all() and torch.equal(y[2, 0].cpu(), torch.zeros(128))
    assert torch.isnan(y[1, 0, 3]) and torch.equal(y[1, 1].cpu(), torch.zeros(128))
    out = gdn.qk_norm_rope_bwd(torch.ones(3, 2, 128, device="cuda"), None, q[:1].expand(3, 2, 128).cuda(), None)
    assert torch.isfinite(out["dq"]).all()


def test_no_tokens_and_one_tensor():
    import gated_delta_rule_112_b200 as gdn
    q, k, w, how = make(0, 2, 1, 64, BF, 32, "rms", True)
    y = gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), **dev(how, w))
    assert y[0].shape == (0, 2, 64)
    out = gdn.qk_norm_rope_bwd(q.cuda(), k.cuda(), q.cuda(), k.cuda(), **dev(how, w))
    assert torch.equal(out["dw_q"].cpu(), torch.zeros(64)) and torch.equal(out["dw_k"].cpu(), torch.zeros(64))
    q, k, w, how = make(4, 2, 0, 64, BF, 32, "rms", True)                   # no heads of k
    y = gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), **dev(how, w))
    assert y[1].shape == (4, 0, 64)
    assert_close("q", np64(y[0]), plain(q, w[0], how).numpy(), tol(BF))
    q, k, w, how = make(5, 2, 1, 64, BF, 32, "rms", True)
    both = gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), **dev(how, w))
    one = gdn.qk_norm_rope_fwd(q.cuda(), None, **{**dev(how, w), "w_k": None})
    assert one[1] is None and torch.equal(one[0], both[0])


def test_captured_replayed_another_stream_and_repeatable():
    import gated_delta_rule_112_b200 as gdn
    q, k, w, how = make(700, 6, 2, 128, BF, 128, "rms", True, seed=70)
    q, k, how = q.cuda(), k.cuda(), dev(how, w)
    dy = [torch.randn(x.shape, device="cuda") for x in (q, k)]
    ref = gdn.qk_norm_rope_fwd(q, k, pack=True, **how)
    rg = gdn.qk_norm_rope_bwd(*dy, q, k, **how)
    again = gdn.qk_norm_rope_bwd(*dy, q, k, **how)
    assert all(torch.equal(rg[n], again[n]) for n in rg)             # sums in a fixed order
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = gdn.qk_norm_rope_fwd(q, k, stream=side, **how)
    g = gdn.qk_norm_rope_bwd(*dy, q, k, stream=side, **how)
    side.synchronize()
    assert torch.equal(y[0], ref[0]) and all(torch.equal(rg[n], g[n]) for n in rg)
    graphs = []
    for _ in range(2):                                               # two graphs, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = gdn.qk_norm_rope_bwd(*dy, *ref[2:], dtype=BF, **how)
        graphs.append((graph, out))
    want = gdn.qk_norm_rope_bwd(*dy, *ref[2:], dtype=BF, **how)
    for _ in range(2):
        for graph, out in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(want[n], out[n]) for n in want)


def test_memory_of_another_streams_inputs_is_kept():
    """Inputs that are given up right after a call on a stream that is still busy: their memory is not handed
    to the next allocation before the call has read it."""
    import gated_delta_rule_112_b200 as gdn
    x = torch.randn(4096, 8, 128, generator=torch.Generator().manual_seed(7)).to(BF)
    ref = gdn.qk_norm_rope_fwd(x.cuda(), None)[0]
    busy = torch.randn(6000, 6000, device="cuda")
    side = torch.cuda.Stream()
    q = x.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):                    # some milliseconds of work ahead of the call
            busy = busy @ busy
            busy /= busy.norm()
    y = gdn.qk_norm_rope_fwd(q, None, stream=side)[0]
    p = gdn.pack(q, stream=side)
    del q
    for _ in range(8):
        torch.empty_like(ref).fill_(float("nan"))
    z = gdn.unpack(p, stream=side)
    side.synchronize()
    assert torch.equal(y, ref)
    assert torch.equal(z.cpu().double(), value(gdn.pack(x.cuda())))


def test_serving_path_together():
    """Projection output -> norms and rotation in place -> the pooled recurrent rule, two calls in a row."""
    import gated_delta_rule_112_b200 as gdn
    T, Hk, Hv, d = 11, 2, 4, 128
    gen = torch.Generator().manual_seed(80)
    wide = torch.randn(T, 2 * Hk * d + Hv * d, generator=gen).to(BF)
    g = -torch.nn.functional.softplus(torch.randn(T, Hv, generator=gen) - 2)
    beta = torch.sigmoid(torch.randn(T, Hv, generator=gen))
    pool = 0.2 * torch.randn(4, Hv, d, d, generator=gen)
    cu, slots = [0, 6, 11], [3, 1]
    f, pos = inv_freq(64), torch.arange(T, dtype=torch.int32) + 50_000
    x = wide.cuda()
    q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([Hk * d, Hk * d, Hv * d], 1))
    gdn.qk_norm_rope_fwd(q, k, positions=pos.cuda(), inv_freq=f.cuda(), q_scale=d ** -0.5, out=(q, k))
    p = pool.cuda()
    o = gdn.recurrent_fwd(q, k, v, g.cuda(), beta.cuda(), p,
                          torch.tensor(slots, dtype=torch.int32, device="cuda"),
                          torch.tensor(cu, dtype=torch.int32, device="cuda"))
    how = dict(norm="l2", positions=pos, inv_freq=f)
    raw = [y.unflatten(1, (-1, d)) for y in wide.split([Hk * d, Hk * d, Hv * d], 1)]
    rq, rk = (plain(raw[0], None, how, d ** -0.5), plain(raw[1], None, how))
    assert_close("q", np64(q), rq.numpy(), tol(BF))
    assert_close("k", np64(k), rk.numpy(), tol(BF))
    for n in range(2):
        rows = slice(cu[n], cu[n + 1])
        qs, ks = (np64(y[rows]).repeat(2, 1)[None] for y in (q, k))     # the rounded rows, as the rule reads them
        ro, rs = oracle.chunk_fwd(qs, ks, np64(v[rows])[None], np64(g[rows])[None], np64(beta[rows])[None],
                                  np64(pool[slots[n]])[None])
        assert_close("o", np64(o[rows]), ro[0], tol(BF))
        assert_close("state", np64(p[slots[n]]), rs[0], TOL_F32)


@pytest.mark.parametrize("exact,bound", [(True, TOL_F32), (False, TOL_BF16)])
def test_training_step_on_the_checkpoint(exact, bound):
    """chunk_fwd_packed / chunk_bwd_packed against the oracle's gradients at the values the checkpoint
    stands for, taken through the norm in fp64. The rows that reach the delta rule are rounded to bf16;
    the reference takes the same rounded rows. dq, dk are stored in bf16: half a step more, and with it
    the rows' rounding in the norm's own chain (another half step)."""
    import gated_delta_rule_112_b200 as gdn
    B, T, H, d = 2, 100, 2, 128
    gen = torch.Generator().manual_seed(90)
    q, k, v = (torch.randn(B, T, H, d, generator=gen).to(BF) for _ in range(3))
    g = -torch.nn.functional.softplus(torch.randn(B, T, H, generator=gen) - 2)
    beta = torch.sigmoid(torch.randn(B, T, H, generator=gen))
    d_o = torch.randn(B, T, H, d, generator=gen).to(BF)
    pos, f = (torch.arange(B * T) % T).to(torch.int32), inv_freq(64)
    how = dict(norm="l2", positions=pos, inv_freq=f)
    c = [x.cuda() for x in (q, k, v, g, beta)]
    o, fs, ck = gdn.chunk_fwd_packed(*c, **dev(how, [None, None]))
    flat = [x.view(B * T, H, d) for x in (q, k)]
    rq, rk = (plain(x, None, how).to(BF).view(B, T, H, d) for x in flat)
    ro, rfs = oracle.chunk_fwd(np64(rq), np64(rk), np64(v), np64(g), np64(beta), None)
    assert_close("o", np64(o), ro, TOL_BF16)
    assert_close("final_state", np64(fs), rfs, TOL_BF16)
    out = gdn.chunk_bwd_packed(ck, c[3], c[4], d_o.cuda(), exact=exact, **dev(how, [None, None]))
    x = [value(y) for y in ck[:3]]
    sq, sk = (gdn.qk_norm_rope_fwd(ck.q, ck.k, **dev(how, [None, None]))[i].view(B, T, H, d) for i in (0, 1))
    ref = oracle.chunk_bwd(np64(sq), np64(sk), x[2].view(B, T, H, d).numpy(), np64(g), np64(beta), np64(d_o), None)
    for n in ("dv", "dg", "dbeta", "d_initial_state"):
        assert_close(n, np64(out[n]), ref[n], bound)
    for i, n in enumerate(("dq", "dk")):
        dx, _ = grads_of(x[i], None, how, 1.0, torch.from_numpy(ref[n]).view(B * T, H, d))
        assert_close(n, np64(out[n]), dx.reshape(B, T, H, d), bound + tol(BF))


def test_angles_are_as_near_at_every_position():
    """Cosines and sines themselves, from rows of (1, 0) pairs, against angles reduced in rational
    arithmetic. The part of a turn, doubled, is at most 1 and is rounded to fp32: 2^-25 half turns, so
    pi 2^-25 rad. Sine and cosine of it are off by one unit in the last place of a value up to 1 at most:
    2^-24. Products with 1 and 0 are exact."""
    from fractions import Fraction
    import gated_delta_rule_112_b200 as gdn
    pi = Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
    gen = torch.Generator().manual_seed(62)
    f = torch.cat([inv_freq(64), torch.tensor([1.5, 37.0, 123.456, 1 / 3], dtype=torch.float64)])
    rows = [torch.randint(lo, hi, (40,), generator=gen) for lo, hi in
            ((0, 1 << 20), (1 << 27, 1 << 28), (1 << 30, (1 << 31) - 1), (-(1 << 31), -(1 << 30)))]
    pos = torch.cat([*rows, torch.tensor([2 ** 31 - 1, -2 ** 31, 0])]).to(torch.int32)
    x = torch.zeros(len(pos), 1, 2 * len(f))
    x[..., 0::2] = 1
    y, _ = gdn.qk_norm_rope_fwd(x.cuda(), None, norm="none", positions=pos.cuda(), inv_freq=f.cuda(),
                                interleaved=True)
    want = torch.empty(len(pos), 2 * len(f), dtype=torch.float64)
    for t, p in enumerate(pos.tolist()):
        for j, w in enumerate(f.tolist()):
            a = p * Fraction(w)
            a = float(a - 2 * pi * round(a / (2 * pi)))
            want[t, 2 * j], want[t, 2 * j + 1] = math.cos(a), math.sin(a)
    assert float((y[:, 0].cpu().double() - want).abs().max()) <= math.pi * 2.0 ** -25 + 2.0 ** -24


def test_smallest_rows_between_the_types():
    """fp32 rows below bf16's range: their codes stand for multiples of 2^-136, exact in fp32 and rounded to
    nearest even in bf16. bf16 rows of that size come back exactly in either type."""
    import gated_delta_rule_112_b200 as gdn
    gen = torch.Generator().manual_seed(63)
    x = torch.randn(64, 3, 96, generator=gen) * torch.exp2(-torch.arange(64.0) / 2 - 110)[:, None, None]
    inexact = 0
    for dtype in (F, BF):
        rows = x.to(dtype)
        p = gdn.pack(rows.cuda())
        codes, scales = plain_pack(rows)
        assert torch.equal(p.scales.cpu(), scales) and torch.equal(p.codes.cpu().double(), codes)
        stands = value(p)
        assert torch.equal(gdn.unpack(p, F).cpu().double(), stands)
        back = gdn.unpack(p).cpu()
        assert torch.equal(back, stands.float().to(BF))       # stands.float() is exact: one rounding
        inexact = int((back.double() != stands).sum())
        assert (inexact > 0) == (dtype == F)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("norm", ["l2", "rms", "none"])
def test_gradients_of_heads_of_one_element(norm, dtype, packed):
    """dx = r dh (1 - h^2), which cancels as eps goes to zero, so each element against r dh. Errors in units of
    2^-24: r 5 (a sum and two products halved, and two units in the last place of the reciprocal root), which
    h^2 has twice; the products x r, x dh and their product 3; w + offset, its product, the last difference and
    product 4: 17, taken as 20. Stored in bf16, half a step of the value more."""
    import gated_delta_rule_112_b200 as gdn
    gen = torch.Generator().manual_seed(64)
    for eps, weights in ((1e-6, False), (1e-6, True), (0.5, True), (0.5, False)):
        q, k = ((2 * torch.randn(h * 7, generator=gen)).to(dtype).view(7, h, 1) for h in (3, 2))
        w = [(1 + 0.3 * torch.randn(1, generator=gen)).to(dtype) if weights else None for _ in "qk"]
        dy = [torch.randn(x.shape, generator=gen) for x in (q, k)]
        how = dict(norm=norm, eps=eps, weight_offset=0.25)
        src = [gdn.pack(x.cuda()) for x in (q, k)] if packed else [q.cuda(), k.cuda()]
        more = dict(dtype=dtype) if packed else {}
        out = gdn.qk_norm_rope_bwd(dy[0].cuda(), dy[1].cuda(), *src, **more, **dev(how, w))
        for i, (x, n) in enumerate(((q, "q"), (k, "k"))):
            x = (value(src[i]) if packed else x).double()
            ref, dw = grads_of(x, w[i], how, 1.0, dy[i])
            r = (x * x + eps).rsqrt() if norm != "none" else torch.ones_like(x)
            dh = dy[i].double() * (w[i].double() + 0.25 if weights else 1.0)
            ref = torch.from_numpy(ref)
            bound = 20 * 2.0 ** -24 * (r * dh).abs()
            if dtype == BF:
                bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
            off = (out["d" + n].cpu().double() - ref).abs()
            assert bool((off <= bound).all()), float((off / bound).max())
            if weights:
                assert_close("dw_" + n, np64(out["dw_" + n]), dw, TOL_F32)


@pytest.mark.parametrize("kind", ["bf16", "bf16_exact", "f32", "short"])
def test_training_step_with_states_weights_and_boundaries(kind):
    """chunk_fwd_packed and chunk_bwd_packed with all that they take: packed sequences (one of them empty) or
    equal ones, initial states, gradients of the final ones, weighted norms, part of the head turned.

    The chunked pass's gradients are held to its own bound b. The norm takes dq through a map whose norm is at
    most q_scale rope_scale max(r |w + offset|), so what b leaves in dq becomes at most that times |dq|; dw sums
    dz h over rows, at most b |dz| times the longest column of h (Cauchy-Schwarz). Roundings of the norm's own
    come on top: tol of the stored type."""
    import gated_delta_rule_112_b200 as gdn
    dtype, d, dv, exact, b = dict(bf16=(BF, 128, 128, False, TOL_BF16), bf16_exact=(BF, 128, 128, True, TOL_F32),
                                  f32=(F, 64, 48, False, TOL_F32), short=(BF, 128, 128, False, TOL_BF16))[kind]
    lens = [1, 1] if kind == "short" else [70, 0, 61]
    cu = None if kind == "short" else torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    B, T, H, N = (2, 1, 3, 2) if kind == "short" else (1, sum(lens), 2, 3)
    gen = torch.Generator().manual_seed(91)
    q, k = (torch.randn(B, T, H, d, generator=gen).to(dtype) for _ in "qk")
    v, d_o = (torch.randn(B, T, H, dv, generator=gen).to(dtype) for _ in "vo")
    g = -torch.nn.functional.softplus(torch.randn(B, T, H, generator=gen) - 2)
    beta = torch.sigmoid(torch.randn(B, T, H, generator=gen))
    s0, ds = (0.3 * torch.randn(N, H, d, dv, generator=gen) for _ in "ab")
    w = [(0.9 + 0.1 * torch.rand(d, generator=gen)).to(dtype) for _ in "qk"]
    how = dict(norm="rms", positions=torch.arange(B * T, dtype=torch.int32) + 77, inv_freq=inv_freq(32),
               weight_offset=float(np.float32(d ** -0.5 - 0.95)),      # keys of about unit length, as the rule wants
               rope_scale=1.1, eps=1e-5)
    scale = [0.5, 1.0]
    kw = dict(dev(how, w), q_scale=scale[0])
    flat = [x.view(B * T, H, d) for x in (q, k)]
    o, fs, ck = gdn.chunk_fwd_packed(*(x.cuda() for x in (q, k, v, g, beta)), s0.cuda(),
                                     None if cu is None else cu.cuda(), **kw)
    rows = [plain(x, y, how, s).to(dtype).view(B, T, H, d) for x, y, s in zip(flat, w, scale)]
    npcu = None if cu is None else cu.numpy()
    ro, rfs = oracle.chunk_fwd(np64(rows[0]), np64(rows[1]), np64(v), np64(g), np64(beta), np64(s0), npcu)
    fwd = TOL_BF16 if dtype == BF else TOL_F32
    assert_close("o", np64(o), ro, fwd)
    assert_close("final_state", np64(fs), rfs, fwd)
    out = gdn.chunk_bwd_packed(ck, g.cuda(), beta.cuda(), d_o.cuda(), s0.cuda(),
                               None if cu is None else cu.cuda(), ds.cuda(), exact=exact, **kw)
    x = [value(y) for y in ck[:3]]
    sq, sk = (np64(y.view(B, T, H, d)) for y in gdn.qk_norm_rope_fwd(ck.q, ck.k, dtype=dtype, **kw))
    ref = oracle.chunk_bwd(sq, sk, x[2].view(B, T, H, dv).numpy(), np64(g), np64(beta), np64(d_o), np64(s0), npcu,
                           np64(ds))
    for n in ("dv", "dg", "dbeta", "d_initial_state"):
        assert_close(n, np64(out[n]), ref[n], b)
    for i, n in enumerate(("dq", "dk")):
        dy = torch.from_numpy(ref[n]).view(B * T, H, d)
        dx, dw = grads_of(x[i], w[i], how, scale[i], dy)
        r = (x[i].detach().square().mean(-1, keepdim=True) + how["eps"]).rsqrt()
        weight, h = w[i].double() + how["weight_offset"], x[i].detach() * r
        dz = scale[i] * how["rope_scale"] * float(dy.norm())
        off = np.linalg.norm(np64(out[n]).reshape(dx.shape) - dx)
        assert off <= b * float((r * weight.abs()).max()) * dz + tol(dtype) * np.linalg.norm(dx), (n, off)
        off = np.linalg.norm(np64(out["dw_" + n[1]]) - dw)
        assert off <= (b + TOL_F32) * dz * float(h.square().sum((0, 1)).max().sqrt()), (n, off)


@pytest.mark.parametrize("weights", [False, True])
def test_gradients_written_over_their_inputs(weights):
    """dq, dk in the place of the raw rows, and in the place of the gradients that they come from."""
    import gated_delta_rule_112_b200 as gdn
    for T, Hq, Hk, d, rot, inter in ((37, 5, 3, 128, 64, False), (2000, 3, 1, 96, 96, True), (9, 7, 2, 33, 2, False)):
        q, k, w, how = make(T, Hq, Hk, d, BF, rot, "l2", weights, inter, seed=65)
        gen = torch.Generator().manual_seed(66)
        dy = [torch.randn(x.shape, generator=gen).to(BF) for x in (q, k)]
        kw = dev(how, w)
        ref = gdn.qk_norm_rope_bwd(dy[0].cuda(), dy[1].cuda(), q.cuda(), k.cuda(), **kw)
        for over in ("rows", "gradients"):
            x, g = [q.cuda(), k.cuda()], [y.cuda() for y in dy]
            into = x if over == "rows" else g
            out = gdn.qk_norm_rope_bwd(*g, *x, out=tuple(into), **kw)
            assert out["dq"].data_ptr() == into[0].data_ptr()
            assert all(torch.equal(out[n], ref[n]) for n in ref if ref[n] is not None)


def test_broadcast_gradients_are_refused():
    import gated_delta_rule_112_b200 as gdn
    q = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(67)).cuda()
    for dy in (torch.ones(6, 1, 64).cuda().expand(6, 2, 64), torch.ones(1, 2, 64).cuda().expand(6, 2, 64)):
        with pytest.raises(gdn.GdnError):
            gdn.qk_norm_rope_bwd(dy, None, q, None)
    with pytest.raises(ValueError):
        gdn.qk_norm_rope_bwd(torch.ones((), device="cuda").expand(6, 2, 64), None, q, None)


def test_rows_of_one_tensor_and_codes_of_the_other():
    """pack=True with an output for q or k alone: the codes of both, the rows of one."""
    import gated_delta_rule_112_b200 as gdn
    q, k, w, how = make(19, 5, 3, 96, BF, 48, "rms", True, seed=68)
    kw = dev(how, w)
    ref = gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), pack=True, **kw)
    for i in range(2):
        out = [None, None]
        out[i] = torch.empty_like((q, k)[i], device="cuda")
        y = gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), pack=True, out=tuple(out), **kw)
        assert torch.equal(y[i], ref[i]) and y[1 - i] is None
        for a, b in zip(y[2:], ref[2:]):
            assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))
            assert torch.equal(a.scales, b.scales)
        with pytest.raises(gdn.GdnError):
            gdn.qk_norm_rope_fwd(q.cuda(), k.cuda(), out=tuple(out), **kw)


def test_training_step_captured_and_on_another_stream():
    """Bit for bit, but for dg and dbeta: the chunkwise backward adds some 20 shares of each token's by atomics in
    any order, which moves their sum by up to 20 units of 2^-24 of the shares (1.2e-6; summed over a chunk's
    tokens for dg, the same of all shares). TOL_F32 leaves a factor of 8 for shares that cancel."""
    import gated_delta_rule_112_b200 as gdn
    gen = torch.Generator().manual_seed(92)
    q, k, v, d_o = (torch.randn(2, 130, 2, 128, generator=gen).to(BF).cuda() for _ in range(4))
    g = -torch.rand(2, 130, 2, generator=gen).cuda()
    beta = torch.rand(2, 130, 2, generator=gen).cuda()

    def step(**how):
        o, fs, ck = gdn.chunk_fwd_packed(q, k, v, g, beta, **how)
        return dict(gdn.chunk_bwd_packed(ck, g, beta, d_o, **how), o=o, fs=fs)

    ref = {n: x.clone() for n, x in step().items() if x is not None}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for n in ref:
        for out in (other, captured):
            if n in ("dg", "dbeta"):
                assert_close(n, np64(out[n]), np64(ref[n]), TOL_F32)
            else:
                assert torch.equal(ref[n], out[n]), n
