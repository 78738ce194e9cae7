"""Host-side refusals of the pooled recurrent rule and of the query/key norms: found before anything is
launched, so no GPU is needed; and the formulas' gradients against differences in fp64."""
import ctypes

import pytest
import torch

import gated_delta_rule_112_b200 as gdn
from gated_delta_rule_112_b200 import build as gbuild

P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn.lib()


def recurrent(L, **kw):
    a = dict(q=P, k=P, v=P, g=P, beta=P, pool=P, slots=P, cu=P, keep=None, reset=None, N=2, T=4, Hk=2, Hv=4,
             dk=128, dv=128, P=8, qs=256, ks=256, vs=512, channel=0, dtype=gdn.BF16, sdt=gdn.F32, o=P,
             status=None)
    a.update(kw)
    return L.gdn_recurrent_fwd(a["q"], a["k"], a["v"], a["g"], a["beta"], a["pool"], a["slots"], a["cu"],
                               a["keep"], a["reset"], a["N"], a["T"], a["Hk"], a["Hv"], a["dk"], a["dv"],
                               a["P"], a["qs"], a["ks"], a["vs"], a["channel"], a["dtype"], a["sdt"], a["o"],
                               a["status"], None)


@pytest.mark.parametrize("bad", [
    dict(dtype=5), dict(sdt=2), dict(Hk=3), dict(Hk=0), dict(N=-1), dict(T=-1), dict(dk=0), dict(dv=0),
    dict(P=-1), dict(cu=None, N=3), dict(slots=None, N=9), dict(qs=255), dict(ks=8), dict(vs=511),
    dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(beta=None), dict(pool=None), dict(o=None),
    dict(pool=ODD), dict(o=ODD), dict(g=ODD), dict(beta=ODD), dict(slots=ODD), dict(cu=ODD), dict(keep=ODD),
    dict(status=ODD), dict(q=ctypes.c_void_p((1 << 20) + 1)),
])
def test_recurrent_refuses(L, bad):
    assert recurrent(L, **bad) == gdn.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(dk=129, qs=512, ks=512), dict(dv=132, vs=600), dict(dv=126),
                                 dict(N=1 << 29)])
def test_recurrent_unsupported(L, bad):
    assert recurrent(L, **bad) == gdn.ERR_UNSUPPORTED


def test_recurrent_without_work(L):
    assert recurrent(L, N=0, T=0, slots=None) == gdn.OK
    assert recurrent(L, T=0) == gdn.OK


def rows(p=1 << 20, ts=1 << 16, hs=128):
    return gdn._Rows(p, ts, hs)


def params(**kw):
    a = dict(T=4, H_q=2, H_k=2, d=128, rot=64, interleaved=0, norm=gdn.NORM_L2, dtype=gdn.BF16, eps=1e-6,
             weight_offset=0.0, q_scale=1.0, rope_scale=1.0, positions=1 << 20, inv_freq=1 << 20, w_q=None,
             w_k=None)
    a.update(kw)
    return gdn._QkParams(**a)


BAD_PARAMS = [dict(dtype=3), dict(T=-1), dict(H_q=-1), dict(H_k=-1), dict(d=0), dict(rot=63), dict(rot=-2),
              dict(rot=130), dict(norm=3), dict(norm=-1), dict(positions=None), dict(inv_freq=None),
              dict(positions=(1 << 20) + 2), dict(inv_freq=(1 << 20) + 4), dict(w_q=(1 << 20) + 1)]


@pytest.mark.parametrize("bad", BAD_PARAMS)
def test_norm_refuses_parameters(L, bad):
    p, r, k8 = params(**bad), ctypes.byref(rows()), ctypes.byref(gdn._PackedRows(1 << 20, 1 << 20))
    pp = ctypes.byref(p)
    assert L.gdn_qk_norm_rope_fwd(pp, r, r, r, r, None, None, None) == gdn.ERR_INVALID_ARG
    assert L.gdn_qk_norm_rope_fwd_packed(pp, k8, k8, r, r, None) == gdn.ERR_INVALID_ARG
    assert L.gdn_qk_norm_rope_bwd(pp, r, r, gdn.F32, r, r, r, r, P, P, P, 1 << 30, None) == gdn.ERR_INVALID_ARG
    assert L.gdn_qk_norm_rope_bwd_packed(pp, r, r, gdn.F32, k8, k8, r, r, P, P, P, 1 << 30,
                                         None) == gdn.ERR_INVALID_ARG


def test_norm_refuses_rows(L):
    good, p = ctypes.byref(rows()), ctypes.byref(params())
    k8 = ctypes.byref(gdn._PackedRows(1 << 20, 1 << 20))
    for bad in (rows(None), rows((1 << 20) + 1), rows(hs=127), rows(ts=255), rows(ts=128, hs=511),
                rows(ts=1 << 40, hs=1 << 28)):
        b = ctypes.byref(bad)
        assert L.gdn_qk_norm_rope_fwd(p, b, good, good, good, None, None, None) == gdn.ERR_INVALID_ARG
        assert L.gdn_qk_norm_rope_fwd(p, good, good, good, b, None, None, None) == gdn.ERR_INVALID_ARG
        assert L.gdn_qk_norm_rope_bwd(p, b, good, gdn.F32, good, good, good, good, None, None, None, 0,
                                      None) == gdn.ERR_INVALID_ARG
        assert L.gdn_qk_norm_rope_bwd(p, good, good, gdn.F32, good, good, good, b, None, None, None, 0,
                                      None) == gdn.ERR_INVALID_ARG
    assert L.gdn_qk_norm_rope_fwd(p, None, good, good, good, None, None, None) == gdn.ERR_INVALID_ARG
    assert L.gdn_qk_norm_rope_fwd(p, good, good, None, good, None, None, None) == gdn.ERR_INVALID_ARG
    for bad8 in (gdn._PackedRows(None, 1 << 20), gdn._PackedRows(1 << 20, None)):
        assert L.gdn_qk_norm_rope_fwd_packed(p, ctypes.byref(bad8), k8, good, good, None) == gdn.ERR_INVALID_ARG
    assert L.gdn_qk_norm_rope_fwd(p, good, good, good, good,
                                  ctypes.byref(gdn._PackedRows(1 << 20, None)), None, None) == gdn.ERR_INVALID_ARG


def test_norm_unsupported_and_workspace(L):
    r = ctypes.byref(rows(hs=300))
    assert L.gdn_qk_norm_rope_fwd(ctypes.byref(params(d=257)), r, r, r, r, None, None, None) == gdn.ERR_UNSUPPORTED
    f = ctypes.byref(params(dtype=gdn.F32))
    assert L.gdn_qk_norm_rope_bwd(f, r, r, gdn.BF16, r, r, r, r, None, None, None, 0, None) == gdn.ERR_UNSUPPORTED
    p = ctypes.byref(params())
    assert L.gdn_qk_norm_rope_bwd(p, r, r, 7, r, r, r, r, None, None, None, 0, None) == gdn.ERR_INVALID_ARG
    # weights and their gradients come together, with a workspace
    assert L.gdn_qk_norm_rope_bwd(p, r, r, gdn.F32, r, r, r, r, P, None, P, 1 << 30, None) == gdn.ERR_INVALID_ARG
    w = ctypes.byref(params(w_q=1 << 20))
    assert L.gdn_qk_norm_rope_bwd(w, r, r, gdn.F32, r, r, r, r, None, None, P, 1 << 30, None) == gdn.ERR_INVALID_ARG
    assert L.gdn_qk_norm_rope_bwd(w, r, r, gdn.F32, r, r, r, r, P, None, None, 1 << 30, None) == gdn.ERR_WORKSPACE
    assert L.gdn_qk_norm_rope_bwd_workspace_size(p) == 0


def test_norm_without_work(L):
    p, r = ctypes.byref(params(T=0, positions=None, inv_freq=None)), ctypes.byref(rows())
    assert L.gdn_qk_norm_rope_fwd(p, r, r, r, r, None, None, None) == gdn.OK
    assert L.gdn_qk_norm_rope_fwd(p, None, None, None, None, None, None, None) == gdn.OK


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 2, 128)
    with pytest.raises(ValueError):
        gdn.qk_norm_rope_fwd(x, x)
    with pytest.raises(ValueError):
        gdn.recurrent_fwd(x, x, x, x[..., 0], x[..., 0], torch.zeros(2, 2, 128, 128))


@pytest.mark.parametrize("norm", ["l2", "rms", "none"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_formula_gradients_against_differences(norm, interleaved):
    """dx = r (dh - h (dh . h) / n) and dw, with the rotation undone, against central differences, fp64:
    step 1e-5, so h^2 and 1e-16 / h both stay below 1e-9 of the gradient's scale."""
    from tests.test_qk_norm_gpu import inv_freq, plain
    gen = torch.Generator().manual_seed(5)
    T, H, d, rot, eps = 2, 2, 12, 8, 1e-2
    x = torch.randn(T, H, d, generator=gen, dtype=torch.float64)
    w = torch.randn(d, generator=gen, dtype=torch.float64)
    dy = torch.randn(T, H, d, generator=gen, dtype=torch.float64)
    how = dict(norm=norm, eps=eps, interleaved=interleaved, inv_freq=inv_freq(rot), rope_scale=1.2,
               positions=torch.tensor([3, 77], dtype=torch.int32))
    back = dict(norm="none", interleaved=interleaved, inv_freq=inv_freq(rot), rope_scale=1.2,
                positions=-how["positions"])
    n = d if norm == "rms" else 1
    r = torch.ones(T, H, 1, dtype=torch.float64) if norm == "none" else \
        ((x * x).sum(-1, keepdim=True) / n + eps).rsqrt()
    h, dz = x * r, plain(dy, None, back)
    dw, dh = (dz * h).sum((0, 1)), dz * w
    dx = dh if norm == "none" else r * (dh - h * (dh * h).sum(-1, keepdim=True) / n)
    for a, grad in ((x, dx), (w, dw)):
        num, flat = torch.zeros_like(a), a.view(-1)
        for i in range(flat.numel()):
            old, vals = float(flat[i]), []
            for step in (1e-5, -1e-5):
                flat[i] = old + step
                vals.append(float((plain(x, w, how) * dy).sum()))
            flat[i] = old
            num.view(-1)[i] = (vals[0] - vals[1]) / 2e-5
        assert float((num - grad).norm() / grad.norm()) < 1e-8


def test_norm_refuses_more_heads_than_its_counters_hold(L):
    k8 = ctypes.byref(gdn._PackedRows(1 << 20, 1 << 20))
    for heads in (dict(H_q=2 ** 31 - 1, H_k=0), dict(H_q=2 ** 30, H_k=1), dict(H_q=2 ** 31 - 1, H_k=2 ** 31 - 1)):
        p, r = ctypes.byref(params(T=1, d=1, rot=0, **heads)), ctypes.byref(rows(ts=1 << 40, hs=1))
        assert L.gdn_qk_norm_rope_fwd(p, r, r, r, r, None, None, None) == gdn.ERR_UNSUPPORTED
        assert L.gdn_qk_norm_rope_fwd_packed(p, k8, k8, r, r, None) == gdn.ERR_UNSUPPORTED
        assert L.gdn_qk_norm_rope_bwd(p, r, r, gdn.F32, r, r, r, r, None, None, None, 0,
                                      None) == gdn.ERR_UNSUPPORTED
        assert L.gdn_qk_norm_rope_bwd_packed(p, r, r, gdn.F32, k8, k8, r, r, None, None, None, 0,
                                             None) == gdn.ERR_UNSUPPORTED


class Shaped:
    """What the binding asks of a tensor, without its memory."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.nbytes = shape, dtype, 1 << 40

    def stride(self):
        out, s = [], 1
        for n in reversed(self.shape):
            out.append(s)
            s *= n
        return tuple(reversed(out))

    def numel(self):
        return self.stride()[0] * self.shape[0]

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


def test_binding_refuses_sizes_past_32_bits(L, monkeypatch):
    """Sizes that ctypes would cut to their low 32 bits: 2^32 + 2 tokens would run as 2."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    f32, big = torch.float32, 2 ** 32 + 2
    for T, N, Hk, Hv in ((big, 1, 1, 1), (big, big, 1, 1), (2, 1, big, big), (2 ** 31, 1, 1, 1)):
        with pytest.raises(ValueError):
            gdn.recurrent_fwd(Shaped(T, Hk, 8), Shaped(T, Hk, 8), Shaped(T, Hv, 8), Shaped(T, Hv, dtype=f32),
                              Shaped(T, Hv, dtype=f32), Shaped(N, Hv, 8, 8, dtype=f32), out=Shaped(T, Hv, 8))
    how = (torch.bfloat16, None, None, None, None, "l2", 1e-6, False, 0.0, 1.0, 1.0)
    for qs, ks in (((big, 1, 8), None), ((2, big, 8), None), ((2, 1, big), None), ((2, 1, 8), (2, big, 8))):
        with pytest.raises(ValueError):
            gdn._qk_params("norm", 0, qs, ks, *how)


class Strided(Shaped):
    """Fewer bytes of memory than its elements would take, as an expanded tensor's."""

    def is_contiguous(self):
        return False


def test_binding_refuses_memory_in_pieces_to_write_to(L, monkeypatch):
    """An expanded workspace or status block counts more bytes than it has."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    f32 = torch.float32
    with pytest.raises(ValueError):
        gdn.recurrent_fwd(Shaped(2, 1, 8), Shaped(2, 1, 8), Shaped(2, 1, 8), Shaped(2, 1, dtype=f32),
                          Shaped(2, 1, dtype=f32), Shaped(2, 1, 8, 8, dtype=f32), out=Shaped(2, 1, 8),
                          status=Strided(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gdn._scratch("norm", Strided(1 << 20, dtype=torch.uint8), 1 << 20, 0)
    with pytest.raises(ValueError):
        gdn._scratch("norm", Shaped(1 << 20, dtype=torch.uint8), 1 << 20, 1)
    assert gdn._scratch("norm", Shaped(1 << 20, dtype=torch.uint8), 1 << 20, 0)
    assert not gdn._scratch("norm", None, 1 << 20, 0)
    codes, scales = Shaped(6, 2, 128, dtype=torch.float8_e4m3fn), Shaped(6, 2, 4, dtype=torch.uint8)
    ckpt = gdn.Checkpoint(*[gdn.Packed(codes, scales)] * 3, (1, 6, 2, 128, 128), torch.bfloat16)
    with pytest.raises(ValueError):
        gdn.chunk_bwd_packed(ckpt, None, None, None, workspace=Strided(1 << 30, dtype=torch.uint8))


@pytest.mark.gpu
def test_workspaces_on_the_gpu(L):
    """What the binding takes and refuses as a workspace, with real tensors."""
    gen = torch.Generator().manual_seed(1)
    q, k, dy = (torch.randn(5, 2, 64, generator=gen).to(torch.bfloat16).cuda() for _ in range(3))
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    ref = gdn.qk_norm_rope_bwd(dy, dy, q, k, w_q=w, w_k=w)
    need = 1 << 20
    ok = gdn.qk_norm_rope_bwd(dy, dy, q, k, w_q=w, w_k=w,
                              workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(ref[n], ok[n]) for n in ref)
    one = torch.zeros(1, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        gdn.qk_norm_rope_bwd(dy, dy, q, k, w_q=w, w_k=w, workspace=one.expand(need))
    assert int(one) == 0


STEP_BAD = [dict(v=(2, 3, 2, 128, "f32")), dict(k=(2, 3, 4, 64, "bf16")), dict(k=(3, 2, 2, 128, "bf16")),
            dict(beta=(2, 3, 2, "bf16")), dict(beta=(2, 3, 1, "f32")), dict(g=(2, 3, 2, "bf16")), dict(g=None),
            dict(initial_state=(1, 2, 128, 128, "f32")), dict(initial_state=(2, 2, 128, 128, "bf16")),
            dict(cu_seqlens=(3, "i64")), dict(d_o=(2, 3, 2, 64, "bf16")), dict(d_o=(2, 3, 2, 128, "f32")),
            dict(d_final_state=(2, 1, 128, 128, "f32"))]


@pytest.mark.parametrize("bad", STEP_BAD)
def test_training_step_refuses_what_it_would_misread(L, monkeypatch, bad):
    """Tensors of another type or fewer elements than the chunked passes would read."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    types = dict(f32=torch.float32, bf16=torch.bfloat16, i64=torch.int64)
    a = dict(q=(2, 3, 2, 128, "bf16"), k=(2, 3, 2, 128, "bf16"), v=(2, 3, 2, 128, "bf16"), g=(2, 3, 2, "f32"),
             beta=(2, 3, 2, "f32"), d_o=(2, 3, 2, 128, "bf16"))
    a = {n: s and Shaped(*s[:-1], dtype=types[s[-1]]) for n, s in {**a, **bad}.items()}
    d_o, more = a.pop("d_o"), {n: a.pop(n) for n in list(a) if n in ("initial_state", "cu_seqlens")}
    last = {n: a.pop(n) for n in list(a) if n == "d_final_state"}
    if not ({"d_o", "d_final_state"} & bad.keys()):
        with pytest.raises(ValueError):
            gdn.chunk_fwd_packed(**a, **more)
    if not ({"q", "k", "v"} & bad.keys()):
        p = gdn.Packed(Shaped(6, 2, 128, dtype=torch.float8_e4m3fn), Shaped(6, 2, 4, dtype=torch.uint8))
        ckpt = gdn.Checkpoint(p, p, p, (2, 3, 2, 128, 128), torch.bfloat16)
        with pytest.raises(ValueError):
            gdn.chunk_bwd_packed(ckpt, a["g"], a["beta"], d_o, **more, **last)


@pytest.mark.parametrize("N,Hv,ok", [(1 << 21, 1, True), ((1 << 21) + 1, 1, False), (1 << 29, 1, False),
                                     (370_727, 32, True), (370_728, 32, False)])
def test_recurrent_refuses_a_search_without_end(L, N, Hv, ok):
    """Every run reads all slots: half a thousand million of them would keep the GPU for days. T = 0 or no
    slots leave nothing to search."""
    how = dict(N=N, Hv=Hv, Hk=1, P=N, vs=128 * Hv, dk=128, dv=4)
    code = recurrent(L, **how, T=0, cu=P)
    assert code == (gdn.OK if ok else gdn.ERR_UNSUPPORTED)
    assert recurrent(L, **how, T=0, cu=P, slots=None) == gdn.OK
