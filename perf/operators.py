"""Cases for the operators around a gated delta layer: the recurrent rule on a pool of states, the
per-head norms of queries and keys with the position rotation, and the 8-bit checkpoint of them.

A case names its operator in "op":

  "recurrent"   runs of new tokens of many sequences against a pool of states, updated in place
  "norm"        per-head norm and rotation of q and k
  "norm_bwd"    its gradients
  "save"        the norm and rotation, keeping q and k in 8 bits for the backward pass
  "restore"     the normed and rotated q and k again, from the 8-bit checkpoint
  "bwd8"        the gradients from the 8-bit checkpoint

`run` computes the plain form in elementary torch operations; with `own` set it makes the library's calls.
"""
import math
import random

import torch

own = False

BLOCK = 32          # elements that share a scale of the 8-bit checkpoint
E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one request being answered: one token of one sequence, the smallest call of a server
        dict(name="step_n1_h16", op="recurrent", n=1, lo=1, hi=1, hk=16, hv=16, dk=128, dv=128,
             dtype="bf16", pool="f32", gate="scalar", spare=7, partial=False, fused=True, lens=1),
        # a full decoding batch on a pool with some free slots
        dict(name="step_n256_h32", op="recurrent", n=256, lo=1, hi=1, hk=32, hv=32, dk=128, dv=128,
             dtype="bf16", pool="f32", gate="scalar", spare=32, partial=False, fused=True, lens=2),
        # a decoding batch with a decay for each channel, states kept in 16 bits, two value heads to a key head
        dict(name="step_n96_channel_bf16pool", op="recurrent", n=96, lo=1, hi=1, hk=16, hv=32, dk=128,
             dv=128, dtype="bf16", pool="bf16", gate="channel", spare=9, partial=False, fused=True, lens=3),
        # drafted tokens being checked: short ragged runs of which the state keeps only the accepted part
        dict(name="verify_n64_l1_6", op="recurrent", n=64, lo=1, hi=6, hk=8, hv=32, dk=128, dv=128,
             dtype="bf16", pool="f32", gate="scalar", spare=11, partial=True, fused=True, lens=4),
        # short prompts and continued ones on odd head sizes, fp32 activations
        dict(name="runs_n13_l0_64_odd", op="recurrent", n=13, lo=0, hi=64, hk=5, hv=15, dk=96, dv=80,
             dtype="f32", pool="f32", gate="scalar", spare=3, partial=True, fused=False, lens=5),
        # the norms of one decoding batch far into long contexts: weighted norm, part of the head rotated
        dict(name="norm_t64_decode", op="norm", t=64, hq=16, hk=16, d=128, rot=64, interleaved=False,
             norm="rms", weights=True, dtype="bf16", far=True, fused=True),
        # the norms of a training batch of the b4h16t4096 configuration
        dict(name="norm_t16384", op="norm", t=16384, hq=16, hk=16, d=128, rot=128, interleaved=False,
             norm="l2", weights=False, dtype="bf16", far=False, fused=True),
        # their gradients, from the fp32 gradients that the chunkwise backward pass gives
        dict(name="norm_bwd_t16384", op="norm_bwd", t=16384, hq=16, hk=16, d=128, rot=128,
             interleaved=False, norm="l2", weights=False, dtype="bf16", grad="f32", far=False, fused=True),
        # weighted norms with fewer key heads, an odd count of tokens and an odd head size
        dict(name="norm_bwd_t4097_odd", op="norm_bwd", t=4097, hq=12, hk=3, d=80, rot=40,
             interleaved=True, norm="rms", weights=True, dtype="bf16", grad="bf16", far=True, fused=False),
        # a training step that keeps q and k in 8 bits: forward ...
        dict(name="save_t16384", op="save", t=16384, hq=16, hk=16, d=128, rot=128, interleaved=False,
             norm="l2", weights=False, dtype="bf16", far=False, fused=True),
        # ... the operands of the chunkwise backward pass again, on a ragged batch ...
        dict(name="restore_t9001", op="restore", t=9001, hq=16, hk=8, d=96, rot=48, interleaved=True,
             norm="rms", weights=True, dtype="bf16", far=True, fused=False),
        # ... and the gradients of the projections' outputs
        dict(name="bwd8_t16384", op="bwd8", t=16384, hq=16, hk=16, d=128, rot=128, interleaved=False,
             norm="rms", weights=True, dtype="bf16", grad="f32", far=False, fused=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["recurrent", "recurrent", "norm", "norm_bwd", "save", "restore", "bwd8"])
    if op == "recurrent":
        kind = rng.choice(["step", "verify", "runs"])
        n = _log(rng, 1, {"step": 256, "verify": 96, "runs": 24}[kind])
        lo, hi = {"step": (1, 1), "verify": (1, rng.randint(2, 9)), "runs": (0, rng.randint(10, 64))}[kind]
        hk = _log(rng, 1, 16)
        dk, dv = (128, 128) if rng.random() < 0.5 else (rng.randint(4, 32) * 4, rng.randint(4, 32) * 4)
        return dict(op=op, n=n, lo=lo, hi=hi, hk=hk, hv=hk * rng.choice([1, 2]), dk=dk, dv=dv,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), pool=rng.choice(["f32", "f32", "bf16"]),
                    gate=rng.choice(["scalar", "scalar", "channel"]), spare=rng.randint(0, 40),
                    partial=kind != "step", fused=rng.random() < 0.5, lens=rng.randrange(1 << 20))
    d = 128 if rng.random() < 0.4 else rng.randint(8, 64) * 4
    rot = rng.choice([0, d // 2, d // 4 * 2, d])
    hq = _log(rng, 1, 32)
    hk = max(1, hq // rng.choice([1, 1, 2, 4]))
    c = dict(op=op, t=_log(rng, 1, min(16384, 16384 * 32 * 128 // ((hq + hk) * d))), hq=hq, hk=hk, d=d,
             rot=rot - rot % 2, interleaved=rng.random() < 0.5, norm=rng.choice(["l2", "rms", "none"]),
             weights=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]), far=rng.random() < 0.5,
             fused=rng.random() < 0.5)
    if op in ("norm_bwd", "bwd8"):
        c["grad"] = rng.choice(["f32", "bf16"]) if c["dtype"] == "bf16" else "f32"
    return c


# ---------------------------------------------------------------- inputs

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _lens(c):
    """Lengths of the runs and how many tokens of each the state keeps: part of the case, not of the seed."""
    r = random.Random(c["lens"])
    lens = [r.randint(c["lo"], c["hi"]) for _ in range(c["n"])]
    keep = [r.randint(0, x) if c["partial"] and r.random() < 0.7 else x for x in lens]
    fresh = [c["partial"] and r.random() < 0.2 for _ in lens]      # new sequences: their state starts at zero
    return lens, keep, fresh


def _split(g, t, heads, fused, dtype):
    """Normal values [t, h, d] for each (h, d): slices of one projection's output, or tensors of their own."""
    if fused:
        x = torch.randn(t, sum(h * d for h, d in heads), generator=g, device="cuda").to(dtype)
        return [y.unflatten(1, hd) for y, hd in zip(x.split([h * d for h, d in heads], 1), heads)]
    return [torch.randn(t, h, d, generator=g, device="cuda").to(dtype) for h, d in heads]


def _inv_freq(c):
    """Rotation frequencies in 64 bits; far positions use ones stretched by 8, as long contexts do."""
    f = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / max(c["rot"], 1))
    return f / 8 if c["far"] else f


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    if c["op"] == "recurrent":
        return _prepare_recurrent(c, g)
    dtype = _type(c["dtype"])
    q, k = _split(g, c["t"], [(c["hq"], c["d"]), (c["hk"], c["d"])], c["fused"], dtype)
    s = dict(c=c, q=q, k=k, wq=None, wk=None, positions=None, inv_freq=None, eps=1e-6,
             q_scale=c["d"] ** -0.5, rope_scale=1.1 if c["far"] else 1.0, offset=0.0)
    if c["weights"]:
        s["wq"], s["wk"] = (((1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(dtype)) for _ in "qk")
    if c["rot"]:
        s["inv_freq"] = _inv_freq(c)
        p = torch.randint(0, 131072, (c["t"],), generator=g, device="cuda") if c["far"] else \
            torch.arange(c["t"], device="cuda") % 4096
        s["positions"] = p.to(torch.int32)
    if c["op"] in ("restore", "bwd8"):
        s["q8"], s["k8"] = _pack(q), _pack(k)
        del s["q"], s["k"]
    if c["op"] in ("norm_bwd", "bwd8"):
        s["dq"], s["dk"] = (torch.randn(c["t"], h, c["d"], generator=g, device="cuda").to(_type(c["grad"]))
                            for h in (c["hq"], c["hk"]))
    return s


def _prepare_recurrent(c, g):
    lens, keep, fresh = _lens(c)
    t, n, dtype = sum(lens), c["n"], _type(c["dtype"])
    slots = n + c["spare"]
    q, k, v = _split(g, t, [(c["hk"], c["dk"]), (c["hk"], c["dk"]), (c["hv"], c["dv"])], c["fused"], dtype)
    for x in (q, k):                                     # as the layer's norm leaves them
        x.copy_(x.float() / x.float().norm(dim=-1, keepdim=True).clamp_min(1e-6))
    gate = (t, c["hv"], c["dk"]) if c["gate"] == "channel" else (t, c["hv"])
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(c=c, q=q, k=k, v=v, longest=max(lens),
             g=-torch.nn.functional.softplus(torch.randn(gate, generator=g, device="cuda") - 2),
             beta=torch.sigmoid(torch.randn(t, c["hv"], generator=g, device="cuda")),
             pool=(0.1 * torch.randn(slots, c["hv"], c["dk"], c["dv"], generator=g, device="cuda")).to(_type(c["pool"])),
             slots=torch.randperm(slots, generator=g, device="cuda")[:n].to(torch.int32),
             cu=None, keep=None, reset=None)
    if c["hi"] > 1:
        s["cu"] = ints([sum(lens[:i]) for i in range(n + 1)])
    if c["partial"]:
        s["keep"], s["reset"] = ints(keep), torch.tensor(fresh, dtype=torch.bool, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        return _run_own(s, op)
    if op == "recurrent":
        return _recurrent(s)
    if op in ("norm", "save"):
        out = dict(q=_norm_rope(s, s["q"], s["wq"], s["q_scale"]), k=_norm_rope(s, s["k"], s["wk"], 1.0))
        if op == "save":
            out["q_codes"], out["q_scales"] = _pack(s["q"])
            out["k_codes"], out["k_scales"] = _pack(s["k"])
        return out
    if op == "restore":
        t = _type(s["c"]["dtype"])
        return dict(q=_norm_rope(s, _unpack(*s["q8"]), s["wq"], s["q_scale"]).to(t),
                    k=_norm_rope(s, _unpack(*s["k8"]), s["wk"], 1.0).to(t))
    q, k = (s["q"], s["k"]) if op == "norm_bwd" else (_unpack(*s["q8"]), _unpack(*s["k8"]))
    dq, dwq = _norm_rope_bwd(s, q, s["dq"], s["wq"], s["q_scale"])
    dk, dwk = _norm_rope_bwd(s, k, s["dk"], s["wk"], 1.0)
    return dict(dq=dq, dk=dk, dw_q=dwq, dw_k=dwk)


def _run_own(s, op):
    import gated_delta_rule_112_b200 as gdn
    if op == "recurrent":
        o = gdn.recurrent_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], slots=s["slots"],
                              cu_seqlens=s["cu"], keep=s["keep"], reset=s["reset"])
        return dict(o=o, pool=s["pool"])
    c = s["c"]
    how = dict(w_q=s["wq"], w_k=s["wk"], positions=s["positions"], inv_freq=s["inv_freq"], norm=c["norm"],
               eps=s["eps"], interleaved=c["interleaved"], weight_offset=s["offset"], q_scale=s["q_scale"],
               rope_scale=s["rope_scale"])
    if op == "norm":
        q, k = gdn.qk_norm_rope_fwd(s["q"], s["k"], **how)
        return dict(q=q, k=k)
    if op == "save":
        q, k, q8, k8 = gdn.qk_norm_rope_fwd(s["q"], s["k"], pack=True, **how)
        return dict(q=q, k=k, q_codes=q8.codes, q_scales=q8.scales, k_codes=k8.codes, k_scales=k8.scales)
    if op == "restore":
        q, k = gdn.qk_norm_rope_fwd(s["q8"], s["k8"], dtype=_type(c["dtype"]), **how)
        return dict(q=q, k=k)
    if op == "norm_bwd":
        return gdn.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], **how)
    return gdn.qk_norm_rope_bwd(s["dq"], s["dk"], s["q8"], s["k8"], dtype=_type(c["dtype"]), **how)


# ---------------------------------------------------------------- plain forms

def _recurrent(s):
    """Token by token, all runs at once: S <- a S (I - b k k^T) + b v k^T, o = S q. The pool holds S^T."""
    c, pool, slots = s["c"], s["pool"], s["slots"].long()
    n, t, rep = c["n"], s["q"].shape[0], c["hv"] // c["hk"]
    start = s["cu"][:-1].long() if s["cu"] is not None else torch.arange(n, device="cuda")
    lens = (s["cu"][1:] - s["cu"][:-1]).long() if s["cu"] is not None else torch.ones_like(start)
    keep = s["keep"].long() if s["keep"] is not None else lens
    S = pool[slots].float()
    if s["reset"] is not None:
        S = torch.where(s["reset"][:, None, None, None], torch.zeros_like(S), S)
    old, kept = pool[slots], S
    o = torch.zeros(t, c["hv"], c["dv"], device="cuda", dtype=s["v"].dtype)
    for i in range(s["longest"]):
        at = (start + i).clamp_max(t - 1)
        on = i < lens
        q, k = (x[at].float().repeat_interleave(rep, 1) for x in (s["q"], s["k"]))
        v, b = s["v"][at].float(), s["beta"][at]
        a = s["g"][at].exp()
        a = a[..., None, None] if a.dim() == 2 else a[..., None]          # on the key axis
        D = S * a
        u = b[..., None] * (v - (D * k[..., None]).sum(-2))
        S = torch.where(on[:, None, None, None], D + k[..., None] * u[..., None, :], S)
        y = (S * q[..., None]).sum(-2)
        o[at[on]] = y[on].to(o.dtype)
        if s["keep"] is not None:
            kept = torch.where((i < keep)[:, None, None, None], S, kept)
    kept = S if s["keep"] is None else kept
    wrote = (keep > 0)[:, None, None, None]               # a run that keeps nothing leaves its slot alone
    pool[slots] = torch.where(wrote, kept.to(pool.dtype), old)
    return dict(o=o, pool=pool)


def _cos_sin(s):
    a = s["positions"].double()[:, None] * s["inv_freq"]
    return (f(a).mul(s["rope_scale"]).float()[:, None] for f in (torch.cos, torch.sin))


def _pairs(c, x):
    r = c["rot"]
    return (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])


def _rotate(s, x, sign):
    c = s["c"]
    if not c["rot"]:
        return x
    cos, sin = _cos_sin(s)
    a, b = _pairs(c, x)
    y = x.clone()
    ya, yb = _pairs(c, y)
    ya.copy_(a * cos - sign * b * sin)
    yb.copy_(b * cos + sign * a * sin)
    return y


def _rnorm(s, x):
    """1 / norm of each head's row, [t, h, 1]."""
    kind, e = s["c"]["norm"], s["eps"]
    if kind == "none":
        return torch.ones_like(x[..., :1])
    ss = (x * x).sum(-1, keepdim=True)
    return 1 / torch.sqrt((ss if kind == "l2" else ss / x.shape[-1]) + e)


def _norm_rope(s, x, w, scale):
    t, x = x.dtype, x.float()
    z = x * _rnorm(s, x)
    if w is not None:
        z = z * (w.float() + s["offset"])
    return (_rotate(s, z, 1) * scale).to(t)


def _norm_rope_bwd(s, x, dy, w, scale):
    kind, t, x = s["c"]["norm"], _type(s["c"]["dtype"]), x.float()
    r = _rnorm(s, x)
    h = x * r
    dz = _rotate(s, dy.float() * scale, -1)
    dh = dz * (w.float() + s["offset"]) if w is not None else dz
    dw = (dz * h).sum((0, 1)) if w is not None else None
    if kind != "none":
        dot = (dh * h).sum(-1, keepdim=True)
        dh = dh - h * (dot if kind == "l2" else dot / x.shape[-1])
    return (dh * r).to(t), dw


def _blocks(x):
    d = x.shape[-1]
    return torch.nn.functional.pad(x, (0, -d % BLOCK)).unflatten(-1, (-1, BLOCK))


def _power(e):
    """2^e in fp32 for whole e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _pack(x):
    """8-bit codes and the exponents (biased by 127) that each 32 of them share: the smallest power of two
    that takes the block's largest finite value to 448 or less. What is not finite becomes NaN."""
    b = _blocks(x.float())
    fine = b.isfinite()
    top = torch.where(fine, b.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, (e - 9 + (m > E4M3_MAX / 512).int()).clamp_min(-127), -127).to(torch.int32)
    codes = torch.where(fine, b * _power(-e)[..., None], float("nan")).to(torch.float8_e4m3fn)
    return codes.flatten(-2)[..., :x.shape[-1]].contiguous(), (e + 127).to(torch.uint8)


def _unpack(codes, scales):
    e = scales.int() - 127                                # in two steps: 2^-127 is below the normal range
    x = _blocks(codes.float()) * _power(e.clamp_min(-126))[..., None]
    return torch.where((e < -126)[..., None], x / 2, x).flatten(-2)[..., :codes.shape[-1]]


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "recurrent":
        return _exact_recurrent(s)
    how = c["op"]
    if how in ("restore", "bwd8"):
        q, k = (x[0].double() * (x[1].double() - 127).exp2().repeat_interleave(BLOCK, -1)[..., :c["d"]]
                for x in (s["q8"], s["k8"]))
    else:
        q, k = s["q"].double(), s["k"].double()
    if how in ("norm", "save", "restore"):
        out = dict(q=_exact_norm(s, q, s["wq"]) * s["q_scale"], k=_exact_norm(s, k, s["wk"]))
        if how == "save":
            out["q_codes"], out["q_scales"] = _exact_pack(q)
            out["k_codes"], out["k_scales"] = _exact_pack(k)
        return out
    out = {}
    for name, x, w, dy, scale in (("q", q, s["wq"], s["dq"], s["q_scale"]), ("k", k, s["wk"], s["dk"], 1.0)):
        with torch.enable_grad():
            x = x.detach().requires_grad_()
            w = None if w is None else w.double().requires_grad_()
            (_exact_norm(s, x, w) * scale).backward(dy.double())
        out["d" + name], out["dw_" + name] = x.grad, None if w is None else w.grad
    return out


def _exact_norm(s, x, w):
    c = s["c"]
    if c["norm"] != "none":
        n = x.square().sum(-1, keepdim=True) if c["norm"] == "l2" else x.square().mean(-1, keepdim=True)
        x = x / (n + s["eps"]).sqrt()
    if w is not None:
        x = x * (w.double() + s["offset"])
    if not c["rot"]:
        return x
    r = c["rot"]
    turn = torch.polar(torch.full_like(s["inv_freq"], s["rope_scale"]).expand(c["t"], -1).contiguous(),
                       s["positions"].double().outer(s["inv_freq"]))[:, None]
    head = x[..., :r]
    pair = head.unflatten(-1, (-1, 2)) if c["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    out = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    out = out if c["interleaved"] else out.transpose(-1, -2)
    return torch.cat([out.flatten(-2), x[..., r:]], -1)


def _exact_pack(x):
    d = x.shape[-1]
    pad = torch.cat([x, x.new_zeros(*x.shape[:-1], -d % BLOCK)], -1)
    b = pad.reshape(*x.shape[:-1], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / E4M3_MAX))
    e = torch.where(top > E4M3_MAX * e.exp2(), e + 1, torch.where(top <= E4M3_MAX * (e - 1).exp2(), e - 1, e))
    e = e.clamp_min(-127)
    y = b / e.exp2()
    step = (torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3).exp2()   # x + 0: codes of -0 are 0 in value
    return (torch.round(y / step) * step).reshape(pad.shape)[..., :d], (e[..., 0] + 127).to(torch.uint8)


def _exact_recurrent(s):
    """Each run at once: its tokens' writes u solve (I + A) u = b (V - decayed S0 K), A below the diagonal."""
    c = s["c"]
    lens, keep, fresh = _lens(c)
    rep, pool = c["hv"] // c["hk"], s["pool"].double()
    o = torch.zeros(sum(lens), c["hv"], c["dv"], device="cuda", dtype=torch.float64)
    slots, at = s["slots"].tolist(), 0
    for i, n in enumerate(lens):
        rows = slice(at, at + n)
        at += n
        if not n:
            continue
        # [head, token, channel]
        q, k = (x[rows].double().transpose(0, 1).repeat_interleave(rep, 0) for x in (s["q"], s["k"]))
        v, b = s["v"][rows].double().transpose(0, 1), s["beta"][rows].double().t()[..., None]
        g = s["g"][rows].double()
        g = (g if g.dim() == 3 else g[..., None]).transpose(0, 1).cumsum(1)          # [h, n, dk or 1]
        S0 = torch.zeros_like(pool[slots[i]]) if fresh[i] else pool[slots[i]]       # [h, dk, dv]
        low = torch.ones(n, n, device="cuda", dtype=torch.bool).tril()
        far = torch.where(low[None, :, :, None], g[:, :, None] - g[:, None], -math.inf).exp()
        kk, qk = ((x[:, :, None] * k[:, None] * far).sum(-1) for x in (k, q))
        A = b * kk.tril(-1)
        u = torch.linalg.solve_triangular(A + torch.eye(n, device="cuda", dtype=A.dtype),
                                          b * (v - (k * g.exp()) @ S0), upper=False, unitriangular=True)
        o[rows] = ((q * g.exp()) @ S0 + qk @ u).transpose(0, 1)
        if keep[i]:
            m = keep[i]
            end = g[:, m - 1:m]
            pool[slots[i]] = end.exp().transpose(1, 2) * S0 + ((end - g[:, :m]).exp() * k[:, :m]).transpose(1, 2) @ u[:, :m]
    return dict(o=o, pool=pool)


# ---------------------------------------------------------------- work

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "recurrent":
        lens, keep, fresh = _lens(c)
        t, p = sum(lens), 2 if c["pool"] == "bf16" else 4
        moved = sum((n > 0 and not f) + (m > 0) for n, m, f in zip(lens, keep, fresh))
        gate = c["dk"] if c["gate"] == "channel" else 1
        token = e * (2 * c["hk"] * c["dk"] + 2 * c["hv"] * c["dv"]) + 4 * c["hv"] * (gate + 1)
        # S k, the rank-one update and S q for each token and head, and the decay
        return {"bytes": moved * c["hv"] * c["dk"] * c["dv"] * p + t * token + 8 * c["n"],
                "flops": t * c["hv"] * c["dk"] * c["dv"] * 7}
    x = c["t"] * (c["hq"] + c["hk"]) * c["d"]
    b8 = x + c["t"] * (c["hq"] + c["hk"]) * -(-c["d"] // BLOCK)
    dy = x * (4 if c.get("grad") == "f32" else 2)
    bytes_ = {"norm": 2 * x * e, "norm_bwd": 2 * x * e + dy, "save": 2 * x * e + b8, "restore": b8 + x * e,
              "bwd8": b8 + dy + x * e}[c["op"]]
    return {"bytes": bytes_ + (4 * c["t"] if c["rot"] else 0), "flops": x * (16 if "bwd" in c["op"] else 8)}
