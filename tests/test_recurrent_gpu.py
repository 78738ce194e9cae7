"""gdn_recurrent_fwd against the fp64 oracle's token recurrence, run by run.

Tolerances (relative L2): fp32 results TOL_F32; results stored in bf16 also get
half a bf16 step, 2^-8 of each value, which bounds the relative L2 of rounding.
"""
import numpy as np
import pytest
import torch

import oracle
from tests.parity import TOL_F32, assert_close, np64

pytestmark = pytest.mark.gpu


def tol(dtype):
    return TOL_F32 + (torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0.0)


def make(lens, Hk, Hv, dk, dv, dtype=torch.bfloat16, pool_dtype=torch.float32, channel=False,
         spare=3, seed=0, gmean=-2.0, beta_scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    q, k = (torch.nn.functional.normalize(torch.randn(T, Hk, dk, generator=gen), dim=-1).to(dtype)
            for _ in "qk")
    d = dict(q=q, k=k, v=torch.randn(T, Hv, dv, generator=gen).to(dtype),
             g=-torch.nn.functional.softplus(
                 torch.randn((T, Hv, dk) if channel else (T, Hv), generator=gen) + gmean),
             beta=beta_scale * torch.sigmoid(torch.randn(T, Hv, generator=gen)),
             pool=(0.3 * torch.randn(N + spare, Hv, dk, dv, generator=gen)).to(pool_dtype),
             slots=torch.randperm(N + spare, generator=gen)[:N].to(torch.int32),
             cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32))
    d["lens"] = list(lens)
    return d


def reference(d, keep=None, reset=None, slots=None):
    """o [T,Hv,dv] and the pool after the call, fp64, from the oracle run by run."""
    lens = d["lens"]
    q, k, v, g, b, pool = (np64(d[x]) for x in ("q", "k", "v", "g", "beta", "pool"))
    rep = v.shape[1] // q.shape[1]
    q, k = q.repeat(rep, 1), k.repeat(rep, 1)
    fn = oracle.kda_chunk_fwd if g.ndim == 3 else oracle.chunk_fwd
    o = np.zeros_like(v)
    at = 0
    slots = d["slots"].tolist() if slots is None else slots
    out = pool.copy()
    for n, length in enumerate(lens):
        rows = slice(at, at + length)
        at += length
        if length == 0 or slots[n] < 0:
            continue
        s0 = pool[slots[n]][None]
        if reset is not None and reset[n]:
            s0 = np.zeros_like(s0)
        m = length if keep is None else keep[n]
        o[rows] = fn(q[rows][None], k[rows][None], v[rows][None], g[rows][None], b[rows][None],
                     s0)[0][0]
        if m:
            r = slice(rows.start, rows.start + m)
            out[slots[n]] = fn(q[r][None], k[r][None], v[r][None], g[r][None], b[r][None], s0)[1][0]
    return o, out


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def call(d, keep=None, reset=None, slots=None, cu=True, out=None, status=None, stream=None):
    import gated_delta_rule_112_b200 as gdn
    pool = d["pool"].cuda()
    o = gdn.recurrent_fwd(
        *(d[x].cuda() for x in ("q", "k", "v", "g", "beta")), pool,
        slots=d["slots"].cuda() if slots is None else ints(slots),
        cu_seqlens=d["cu"].cuda() if cu else None, keep=None if keep is None else ints(keep),
        reset=None if reset is None else torch.tensor(reset, dtype=torch.bool, device="cuda"),
        out=out, status=status, stream=stream)
    return o, pool


def check(d, o, pool, **how):
    ro, rp = reference(d, **how)
    if ro.size:
        assert_close("o", np64(o), ro, tol(d["v"].dtype))
    assert_close("pool", np64(pool), rp, tol(pool.dtype))


BF, F = torch.bfloat16, torch.float32
CASES = [
    # lens, Hk, Hv, dk, dv, dtype, pool dtype, channel gate
    ([1], 1, 1, 128, 128, BF, F, False),
    ([1] * 7, 2, 2, 128, 128, BF, F, False),
    ([1] * 5, 2, 6, 128, 128, F, F, True),
    ([3, 1, 0, 6, 2], 4, 4, 128, 128, BF, F, False),
    ([9, 8, 7, 17], 1, 4, 128, 128, BF, BF, False),
    ([5, 0, 33], 3, 3, 96, 80, F, F, False),
    ([2, 70], 2, 4, 64, 128, BF, F, True),
    ([4, 5], 1, 2, 36, 20, F, BF, True),
    ([6], 5, 5, 128, 4, F, F, False),
    ([1, 2, 3], 2, 2, 1, 8, F, F, False),
    ([11, 3], 1, 3, 33, 12, BF, F, True),
    ([300, 129], 1, 1, 128, 64, F, F, False),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_runs_match_oracle(case):
    lens, Hk, Hv, dk, dv, dtype, pdt, channel = CASES[case]
    d = make(lens, Hk, Hv, dk, dv, dtype, pdt, channel, seed=case)
    o, pool = call(d)
    check(d, o, pool)
    others = sorted(set(range(d["pool"].shape[0])) - set(d["slots"].tolist()))
    assert torch.equal(pool[others].cpu(), d["pool"][others])       # slots of nobody: untouched


@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("pdt", [F, BF])
def test_keep_and_reset(channel, pdt):
    lens = [6, 6, 6, 1, 12, 0]
    keep, reset = [0, 3, 6, 0, 9, 0], [False, True, False, True, True, True]
    d = make(lens, 2, 4, 128, 128, BF, pdt, channel, seed=20)
    o, pool = call(d, keep=keep, reset=reset)
    check(d, o, pool, keep=keep, reset=reset)
    for n in (0, 3, 5):                                             # nothing kept: bit for bit
        s = d["slots"][n]
        assert torch.equal(pool[s].cpu(), d["pool"][s])


def test_equal_lengths_without_cu_and_without_slots():
    import gated_delta_rule_112_b200 as gdn
    d = make([4] * 3, 2, 2, 128, 128, F, seed=21, spare=0)
    d["slots"] = torch.arange(3, dtype=torch.int32)
    pool = d["pool"].cuda()
    o = gdn.recurrent_fwd(*(d[x].cuda() for x in ("q", "k", "v", "g", "beta")), pool)
    check(d, o, pool)


def test_matches_decode_step():
    import gated_delta_rule_112_b200 as gdn
    for channel, cu in ((False, False), (True, False), (False, True), (True, True)):
        d = make([1] * 6, 3, 3, 128, 128, F, seed=22, channel=channel, spare=0)
        d["slots"] = torch.arange(6, dtype=torch.int32)
        o, pool = call(d, cu=cu)
        state = d["pool"].cuda()
        step = gdn.kda_decode_step if channel else gdn.decode_step
        ref = step(*(d[x].cuda() for x in ("q", "k", "v", "g", "beta")), state)
        assert_close("o", np64(o), np64(ref), TOL_F32)
        assert_close("state", np64(pool), np64(state), TOL_F32)


def test_one_call_equals_two():
    d = make([13, 9], 1, 2, 128, 128, F, seed=23)
    o, pool = call(d)
    import gated_delta_rule_112_b200 as gdn
    p2 = d["pool"].cuda()
    parts = []
    for (a0, b0), (a1, b1) in (((0, 5), (13, 17)), ((5, 13), (17, 22))):   # tokens of each run, call by call
        rows = torch.cat([torch.arange(a0, b0), torch.arange(a1, b1)])
        parts.append((rows, gdn.recurrent_fwd(
            *(d[x][rows].cuda() for x in ("q", "k", "v", "g", "beta")), p2, d["slots"].cuda(),
            ints([0, b0 - a0, len(rows)]))))
    both = torch.empty_like(o)
    for rows, y in parts:
        both[rows.cuda()] = y
    assert_close("o", np64(both), np64(o), TOL_F32)
    assert_close("pool", np64(p2), np64(pool), TOL_F32)


def test_padding_and_tokens_behind_the_last_run_are_left_alone():
    d = make([2, 3, 1], 2, 2, 128, 128, BF, seed=24)
    slots = [int(d["slots"][0]), -1, int(d["slots"][2])]
    extra = 5                                                      # padded rows of a captured batch
    for x in ("q", "k", "v", "g", "beta"):
        d[x] = torch.cat([d[x], torch.full_like(d[x][:1], float("nan")).expand(extra, *d[x].shape[1:])])
    out = torch.full(tuple(d["v"].shape), 7.0, dtype=BF, device="cuda")
    o, pool = call(d, slots=slots, out=out)
    d["lens"], full = [2, 3, 1], d
    ref_o, ref_p = reference({**full, **{x: full[x][:6] for x in ("q", "k", "v", "g", "beta")}}, slots=slots)
    assert torch.equal(o[2:5].cpu(), torch.full_like(o[2:5].cpu(), 7.0))
    assert torch.equal(o[6:].cpu(), torch.full_like(o[6:].cpu(), 7.0))
    assert_close("o", np64(o[:2]), ref_o[:2], tol(BF))
    assert_close("pool", np64(pool), ref_p, TOL_F32)


def test_strided_and_unaligned_inputs():
    import gated_delta_rule_112_b200 as gdn
    for dtype in (BF, F):
        d = make([3, 8], 2, 4, 128, 64, dtype, seed=25)
        T = 11
        for offset in (0, 1):          # slices of one projection output, then off by one element
            wide = torch.zeros(T, offset + 2 * 128 * 2 + 4 * 64 + 5, dtype=dtype, device="cuda")
            q, k, v = (wide[:, offset + a:offset + a + h * w].unflatten(1, (h, w))
                       for a, h, w in ((0, 2, 128), (256, 2, 128), (512, 4, 64)))
            for x, name in ((q, "q"), (k, "k"), (v, "v")):
                x.copy_(d[name])
            pool = d["pool"].cuda()
            o = gdn.recurrent_fwd(q, k, v, d["g"].cuda(), d["beta"].cuda(), pool, d["slots"].cuda(),
                                  d["cu"].cuda())
            check(d, o, pool)
            one = make([1] * T, 2, 4, 128, 64, dtype, seed=35)     # the same rows, one token a run
            pool = one["pool"].cuda()
            o = gdn.recurrent_fwd(q, k, v, d["g"].cuda(), d["beta"].cuda(), pool, one["slots"].cuda())
            check({**one, **{x: d[x] for x in ("q", "k", "v", "g", "beta")}}, o, pool)


@pytest.mark.parametrize("channel", [False, True])
def test_gates_at_their_ends(channel):
    """g = -inf forgets everything (also what was large), strong decays, growth, beta up to 2."""
    d = make([9, 20, 5], 1, 2, 128, 128, F, channel=channel, seed=26, gmean=3.0, beta_scale=2.0)
    d["g"][4] = float("-inf")
    d["g"][11:19] = -60.0             # the running product of decays underflows fp32
    d["g"][29:33] = 1.5               # and a growing state
    d["g"][3] = 0.0
    o, pool = call(d)
    check(d, o, pool)


# One token a run without boundaries has a kernel of its own.
ONE = [
    # N, Hk, Hv, dk, dv, dtype, pool dtype, channel gate
    (1, 1, 1, 128, 128, BF, F, False),
    (5, 2, 6, 128, 128, BF, F, True),
    (7, 3, 3, 128, 128, F, BF, False),
    (4, 2, 4, 128, 128, BF, BF, True),
    (3, 1, 2, 96, 80, BF, F, False),
    (3, 1, 2, 100, 72, F, BF, True),
    (2, 2, 2, 33, 8, BF, BF, False),
    (2, 1, 5, 64, 12, F, F, True),
    (2, 1, 1, 128, 12, F, BF, False),          # rows of a bf16 state that are no whole pieces
    (3, 1, 1, 1, 4, F, F, False),
]


@pytest.mark.parametrize("case", range(len(ONE)))
def test_one_token_a_run(case):
    N, Hk, Hv, dk, dv, dtype, pdt, channel = ONE[case]
    d = make([1] * N, Hk, Hv, dk, dv, dtype, pdt, channel, seed=100 + case, beta_scale=2.0)
    o, pool = call(d, cu=False)
    check(d, o, pool)
    others = sorted(set(range(d["pool"].shape[0])) - set(d["slots"].tolist()))
    assert torch.equal(pool[others].cpu(), d["pool"][others])


@pytest.mark.parametrize("pdt", [F, BF])
@pytest.mark.parametrize("channel", [False, True])
def test_one_token_keep_reset_padding_and_decay_of_zero(pdt, channel):
    d = make([1] * 6, 2, 4, 128, 128, BF, pdt, channel, seed=120)
    d["g"][2] = float("-inf")
    keep, reset = [1, 0, 1, 1, 0, 1], [False, False, False, True, True, False]
    slots = d["slots"].tolist()
    slots[5] = -3
    out = torch.full(tuple(d["v"].shape), 7.0, dtype=BF, device="cuda")
    o, pool = call(d, keep=keep, reset=reset, slots=slots, cu=False, out=out)
    assert torch.equal(o[5].cpu(), torch.full_like(o[5].cpu(), 7.0))
    ro, rp = reference(d, keep=keep, reset=reset, slots=slots)
    assert_close("o", np64(o[:5]), ro[:5], tol(BF))
    assert_close("pool", np64(pool), rp, tol(pdt))
    for n in (1, 4):
        assert torch.equal(pool[slots[n]].cpu(), d["pool"][slots[n]])


@pytest.mark.parametrize("how,spoilt", [
    (dict(slots=[0, 99, 2]), [1]), (dict(slots=[0, 2, 2]), [1, 2]),
    (dict(slots=[0, 2, 2], keep=[1, 0, 1]), [1, 2]), (dict(keep=[1, 2, 1]), [1]),
    (dict(keep=[1, -1, 1]), [1]), (dict(slots=[0, 2, 2], keep=[1, 0, 0]), [])])
def test_one_token_bad_runs(how, spoilt):
    import gated_delta_rule_112_b200 as gdn
    d = make([1] * 3, 1, 2, 128, 128, BF, seed=121)
    d["slots"] = torch.arange(3, dtype=torch.int32)
    status = gdn.status_block()
    o, pool = call(d, status=status, cu=False, **how)
    assert gdn.get_status(status) == (gdn.ERR_INVALID_ARG if spoilt else gdn.OK)
    slots = how.get("slots", [0, 1, 2])
    ro, rp = reference(d, slots=[-1 if n in spoilt else x for n, x in enumerate(slots)],
                       keep=None if "keep" not in how else
                       [0 if n in spoilt else x for n, x in enumerate(how["keep"])])
    for n in range(3):
        if n in spoilt:
            assert torch.isnan(o[n]).all()
        else:
            assert_close(f"o of run {n}", np64(o[n]), ro[n], tol(BF))
    assert_close("pool", np64(pool), rp, TOL_F32)


@pytest.mark.parametrize("cu", [False, True])
def test_more_runs_than_a_grid_dimension(cu):
    """70,000 runs of a tiny state; the last ones checked against the rule in fp64."""
    import gated_delta_rule_112_b200 as gdn
    N = 70_000
    d = make([1] * N, 1, 1, 4, 4, F, seed=122, spare=0)
    status = gdn.status_block()
    o, pool = call(d, cu=cu, status=status)
    assert gdn.get_status(status) == gdn.OK
    q, k, v, g, b = (np64(d[x])[:, 0] for x in ("q", "k", "v", "g", "beta"))
    S = np64(d["pool"])[d["slots"].numpy(), 0] * np.exp(g)[:, None, None]
    u = b[:, None] * (v - np.einsum("nji,nj->ni", S, k))
    S = S + k[:, :, None] * u[:, None]
    assert_close("o", np64(o[:, 0]), np.einsum("nji,nj->ni", S, q), TOL_F32)
    assert_close("pool", np64(pool[d["slots"].long().cuda(), 0]), S, TOL_F32)


def test_two_calls_at_once_on_disjoint_slots():
    import gated_delta_rule_112_b200 as gdn
    d = make([3, 5, 2, 7], 2, 4, 128, 128, BF, seed=123)
    ref, rpool = call(d)
    pool = d["pool"].cuda()
    args = [d[x].cuda() for x in ("q", "k", "v", "g", "beta")]
    outs = []
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(2):
        lo, hi = (0, 8) if rep == 0 else (8, 17)
        cu = ints([0, 3, 8] if rep == 0 else [0, 2, 9])
        slots = d["slots"][2 * rep:2 * rep + 2].cuda()
        part = [x[lo:hi].contiguous() for x in args]
        torch.cuda.synchronize()
        outs.append((part, slots, cu))
    os = [gdn.recurrent_fwd(*p, pool, s, c, stream=st) for (p, s, c), st in zip(outs, streams)]
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(os), ref) and torch.equal(pool, rpool)


def test_large_pool_offsets():
    """Slots whose elements lie past 2^32 bytes and past 2^31 elements."""
    import gated_delta_rule_112_b200 as gdn
    d = make([2, 1], 1, 1, 128, 128, BF, BF, seed=27, spare=0)
    P = 140_000
    pool = torch.empty(P, 1, 128, 128, dtype=BF, device="cuda")
    slots = [P - 1, 131_073]
    pool[slots] = d["pool"].cuda()
    o = gdn.recurrent_fwd(*(d[x].cuda() for x in ("q", "k", "v", "g", "beta")), pool, ints(slots),
                          d["cu"].cuda())
    d["slots"] = torch.arange(2, dtype=torch.int32)
    check(d, o, pool[slots])
    d = make([1, 1], 1, 1, 128, 128, BF, BF, seed=34, spare=0)             # one token a run
    pool[slots] = d["pool"].cuda()
    o = gdn.recurrent_fwd(*(d[x].cuda() for x in ("q", "k", "v", "g", "beta")), pool, ints(slots))
    d["slots"] = torch.arange(2, dtype=torch.int32)
    check(d, o, pool[slots])


BAD = {  # what is wrong with run 1 of three: its arguments, and the runs it spoils
    "slot_past_pool": (dict(slots=[0, 99, 2]), [1]),
    "slot_twice": (dict(slots=[0, 2, 2]), [1, 2]),
    "slot_twice_one_keeps": (dict(slots=[0, 2, 2], keep=[1, 0, 1]), [1, 2]),
    "keep_past_length": (dict(keep=[1, 9, 4]), [1]),
    "keep_negative": (dict(keep=[1, -1, 4]), [1]),
}


@pytest.mark.parametrize("bad", sorted(BAD))
def test_bad_runs_are_refused(bad):
    import gated_delta_rule_112_b200 as gdn
    how, spoilt = BAD[bad]
    d = make([2, 3, 4], 1, 2, 128, 128, BF, seed=28)
    d["slots"] = torch.arange(3, dtype=torch.int32)
    status = gdn.status_block()
    o, pool = call(d, status=status, **how)
    assert gdn.get_status(status) == gdn.ERR_INVALID_ARG
    assert gdn.get_status(status) == gdn.OK                         # read once
    ro, rp = reference(d, slots=[s if n not in spoilt else -1 for n, s in
                                 enumerate(how.get("slots", [0, 1, 2]))],
                       keep=None if "keep" not in how else
                       [0 if n in spoilt else x for n, x in enumerate(how["keep"])])
    cu = d["cu"].tolist()
    for n in range(3):
        rows = slice(cu[n], cu[n + 1])
        if n in spoilt:
            assert torch.isnan(o[rows]).all()
        else:
            assert_close(f"o of run {n}", np64(o[rows]), ro[rows], tol(BF))
    assert_close("pool", np64(pool), rp, TOL_F32)
    assert torch.equal(pool[3:].cpu(), d["pool"][3:])


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [-2, 2, 5, 9], [0, 2, 5, 40]])
def test_bad_boundaries_are_reported(cu):
    import gated_delta_rule_112_b200 as gdn
    d = make([2, 3, 4], 1, 1, 128, 128, F, seed=29)
    d["cu"] = torch.tensor(cu, dtype=torch.int32)
    status = gdn.status_block()
    call(d, status=status)
    assert gdn.get_status(status) == gdn.ERR_INVALID_ARG


def test_runs_that_keep_nothing_may_share_a_slot():
    import gated_delta_rule_112_b200 as gdn
    d = make([2, 3, 4, 0], 1, 2, 128, 128, BF, seed=30)
    status = gdn.status_block()
    o, pool = call(d, slots=[2, 2, 2, 2], keep=[0, 0, 0, 0], status=status)
    assert gdn.get_status(status) == gdn.OK
    check(d, o, pool, slots=[2, 2, 2, 2], keep=[0, 0, 0, 0])
    assert torch.equal(pool.cpu(), d["pool"])


def test_many_runs_each_finds_its_slot():
    """More runs than threads of a block, one slot named twice far apart."""
    import gated_delta_rule_112_b200 as gdn
    d = make([1] * 700, 1, 1, 32, 16, F, seed=31, spare=0)
    slots = d["slots"].tolist()
    status = gdn.status_block()
    o, pool = call(d, status=status)
    assert gdn.get_status(status) == gdn.OK
    check(d, o, pool)
    slots[699] = slots[3]
    o, pool = call(d, slots=slots, status=status)
    assert gdn.get_status(status) == gdn.ERR_INVALID_ARG
    assert torch.isnan(o[[3, 699]]).all() and torch.isfinite(o[4:699]).all()


def test_captured_replayed_and_on_another_stream():
    import gated_delta_rule_112_b200 as gdn
    d = make([3, 1, 4], 2, 4, 128, 128, BF, seed=32)
    ref, rpool = call(d)
    pool = d["pool"].cuda()
    args = [d[x].cuda() for x in ("q", "k", "v", "g", "beta")]
    slots, cu = d["slots"].cuda(), d["cu"].cuda()
    out = torch.empty_like(ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = gdn.recurrent_fwd(*args, pool, slots, cu, stream=side)
    side.synchronize()
    assert torch.equal(o, ref) and torch.equal(pool, rpool)
    pool.copy_(d["pool"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.recurrent_fwd(*args, pool, slots, cu, out=out)
    pool.copy_(d["pool"])
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(pool, rpool)


def test_workload_pool_step_full_size():
    """The decode workload's batch (N=256, H=32, d=128) from a pool, every state and output."""
    d = make([1] * 256, 32, 32, 128, 128, BF, seed=33, spare=8)
    for cu in (False, True):
        o, pool = call(d, cu=cu)
        check(d, o, pool)


def test_padding_runs_may_have_any_boundaries():
    """The unused runs at the end of a captured batch: negative slots with boundaries, keep points and
    resets left over from an earlier batch. They are no error and change nothing."""
    import gated_delta_rule_112_b200 as gdn
    d = make([2, 3], 2, 2, 128, 128, BF, seed=36, spare=5)
    ref, rpool = call(d)
    slots = d["slots"].tolist()
    status = gdn.status_block()
    for tail in ([5, 3, 9], [0, 0, -7], [40, 2, 1 << 30]):
        p = {**d, "cu": torch.tensor([0, 2, 5, *tail], dtype=torch.int32)}
        out = torch.full(tuple(ref.shape), 7.0, dtype=BF, device="cuda")
        o, pool = call(p, slots=[*slots, -1, -5, -1], keep=[2, 3, 9, -4, 1],
                       reset=[False, False, True, True, False], out=out, status=status)
        assert gdn.get_status(status) == gdn.OK
        assert torch.equal(o, ref) and torch.equal(pool, rpool)


# fp32 rows on a bf16 pool: the kernel for runs takes the tokens' updates one by one and fetches later.
STEP = [
    # lens, Hk, Hv, dk, dv, channel gate; runs of three groups of four and more
    ([9, 30, 13], 2, 4, 128, 128, False),
    ([9, 30, 13], 2, 4, 128, 128, True),
    ([17, 0, 12, 21], 1, 2, 33, 12, False),            # rows that are not copied in pieces
    ([17, 0, 12, 21], 1, 2, 33, 12, True),
    ([64, 10], 3, 3, 96, 80, False),
    ([25], 1, 4, 64, 128, True),
]


@pytest.mark.parametrize("part", [False, True])
@pytest.mark.parametrize("case", range(len(STEP)))
def test_fp32_rows_on_a_bf16_pool(case, part):
    lens, Hk, Hv, dk, dv, channel = STEP[case]
    d = make(lens, Hk, Hv, dk, dv, F, BF, channel, seed=200 + case, beta_scale=2.0)
    how = {}
    if part:                                           # keep points inside groups, fresh states
        how = dict(keep=[[6, 5, 0, n][i] if n else 0 for i, n in enumerate(lens)],
                   reset=[i % 2 == 1 for i in range(len(lens))])
    o, pool = call(d, **how)
    check(d, o, pool, **how)


def rounded_update():
    """Twelve tokens on a state of ones: k of token t is (x, -x) in rows 2t and 2t + 1, so S k is zero in any
    order, k_l . k_m is zero and u is v. The rule then stores 1 + v x and 1 - v x, with a rounding of the
    product and one of the sum. Three quarters of the columns hold a v for which one fused rounding of 1 + v x
    ends on the other side of a bf16 border. Returns k, v, the stored state and the fused one."""
    rng = np.random.default_rng(5)
    k, v = np.zeros((12, 128), np.float32), rng.standard_normal((12, 128)).astype(np.float32)
    at = np.float32(2.0 ** -8 + 2.0 ** -24)            # 1 + this is halfway between two fp32 numbers
    for t in range(12):
        found = []
        while not found:
            x = np.float32(rng.uniform(0.4, 0.7))
            w = (np.float64(at) / np.float64(x)).astype(np.float32)
            for u in (np.nextafter(w, np.float32(0)), w, np.nextafter(w, np.float32(1))):
                if u * x == at and np.float64(u) * np.float64(x) > np.float64(at):
                    found.append(u)
        k[t, 2 * t], k[t, 2 * t + 1] = x, -x
        v[t, :96] = np.resize(np.array(found, np.float32), 96)
    one, both = np.float32(1), k.T[:, :, None] * v[None]            # [row, token, column], rounded
    step, fused = np.ones((128, 128), np.float32), np.ones((128, 128), np.float32)
    for j in range(24):
        step[j] = one + both[j, j // 2]
        fused[j] = (1 + np.float64(k[j // 2, j]) * np.float64(v[j // 2])).astype(np.float32)
    to = lambda x: torch.from_numpy(x).to(BF)  # noqa: E731
    return torch.from_numpy(k), torch.from_numpy(v), to(step), to(fused)


@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("one", [False, True])
def test_fp32_rows_on_a_bf16_pool_round_products_and_sums(one, channel):
    """The stored state of a run, and of single tokens, is the rule's own, bit for bit."""
    import gated_delta_rule_112_b200 as gdn
    k, v, step, fused = rounded_update()
    assert int((step != fused).sum()) >= 12 * 96
    n = 12 if one else 1
    pool = torch.ones(n, 1, 128, 128, dtype=BF, device="cuda")
    k, v = k[:, None].cuda(), v[:, None].cuda()
    g = torch.zeros(12, 1, 128, device="cuda") if channel else torch.zeros(12, 1, device="cuda")
    gdn.recurrent_fwd(k, k, v, g, torch.ones(12, 1, device="cuda"), pool, slots=ints(list(range(n))))
    if one:                                            # each token changed its own two rows of its own state
        rows = torch.arange(24)
        assert torch.equal(pool[rows // 2, 0, rows].cpu(), step[:24])
    else:
        assert torch.equal(pool[0, 0].cpu(), step)


def test_calls_repeat_bit_for_bit():
    """One token of one sequence, a batch of them and runs: the same inputs give the same bits."""
    for lens, Hk, Hv, dtype, pdt, cu in (([1], 16, 16, BF, F, False), ([1] * 64, 8, 16, BF, BF, False),
                                         ([3, 17, 1, 6], 2, 4, F, F, True), ([9, 14], 2, 2, F, BF, True)):
        d = make(lens, Hk, Hv, 128, 128, dtype, pdt, seed=210)
        first = call(d, cu=cu)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(call(d, cu=cu), first))


def test_slots_without_boundaries_and_boundaries_without_slots():
    import gated_delta_rule_112_b200 as gdn
    d = make([5] * 4, 2, 4, 128, 128, BF, seed=220, spare=0)         # equal runs: reset, keep and slots
    how = dict(keep=[5, 2, 0, 4], reset=[True, False, True, False])
    o, pool = call(d, cu=False, **how)
    check(d, o, pool, **how)
    d = make([3, 0, 6], 1, 2, 64, 32, F, BF, seed=221, spare=2)
    pool = d["pool"].cuda()
    o = gdn.recurrent_fwd(*(d[x].cuda() for x in ("q", "k", "v", "g", "beta")), pool, cu_seqlens=d["cu"].cuda())
    d["slots"] = torch.arange(3, dtype=torch.int32)
    check(d, o, pool)


def test_no_runs_and_no_tokens():
    import gated_delta_rule_112_b200 as gdn
    d = make([2, 1], 1, 2, 128, 128, BF, seed=222)
    args = [d[x].cuda() for x in ("q", "k", "v", "g", "beta")]
    pool, out = d["pool"].cuda(), torch.full(tuple(d["v"].shape), 7.0, dtype=BF, device="cuda")
    gdn.recurrent_fwd(*args, pool, ints([]), ints([0]), out=out)     # no runs: nothing is touched
    assert bool((out == 7).all()) and torch.equal(pool.cpu(), d["pool"])
    o = gdn.recurrent_fwd(*(x[:0] for x in args), pool, ints([2, 0]), ints([0, 0, 0]))
    assert o.shape == (0, 2, 128) and torch.equal(pool.cpu(), d["pool"])


@pytest.mark.parametrize("lens", [[6, 11], [1] * 5])
def test_gates_off_their_alignment(lens):
    """A channel gate that starts 4 bytes off a 16-byte boundary: read one by one."""
    import gated_delta_rule_112_b200 as gdn
    d = make(lens, 2, 4, 128, 128, BF, channel=True, seed=223)
    wide = torch.zeros(d["g"].numel() + 1, device="cuda")
    g = wide[1:].view(d["g"].shape)
    g.copy_(d["g"])
    pool = d["pool"].cuda()
    o = gdn.recurrent_fwd(*(d[x].cuda() for x in "qkv"), g, d["beta"].cuda(), pool, d["slots"].cuda(),
                          None if len(lens) == 5 else d["cu"].cuda())
    check(d, o, pool)


def test_a_captured_step_replayed_with_other_slots():
    """A server's graph: one token a run, slots, keep and reset changed between replays."""
    import gated_delta_rule_112_b200 as gdn
    d = make([1] * 6, 2, 4, 128, 128, BF, seed=224, spare=6)
    args = [d[x].cuda() for x in ("q", "k", "v", "g", "beta")]
    pool, slots = d["pool"].cuda(), d["slots"].cuda()
    keep, reset = ints([1] * 6), torch.zeros(6, dtype=torch.bool, device="cuda")
    gdn.recurrent_fwd(*args, pool, slots, keep=keep, reset=reset)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gdn.recurrent_fwd(*args, pool, slots, keep=keep, reset=reset)
    for new, k, r in (([11, 0, 3, 7, 5, 2], [1, 0, 1, 1, 1, 0], [0, 0, 1, 0, 1, 1]),
                      ([1, 2, -1, 4, 6, -4], [1, 1, 1, 0, 1, 1], [1, 0, 0, 0, 0, 1])):
        pool.copy_(d["pool"])
        out.fill_(7.0)
        slots.copy_(ints(new))
        keep.copy_(ints(k))
        reset.copy_(ints(r).bool())
        graph.replay()
        torch.cuda.synchronize()
        ro, rp = reference(d, keep=k, reset=r, slots=new)
        on = [i for i in range(6) if new[i] >= 0]
        assert_close("o", np64(out[on]), ro[on], tol(BF))
        assert_close("pool", np64(pool), rp, TOL_F32)
        assert all(bool((out[i] == 7).all()) for i in range(6) if new[i] < 0)
