"""The bounds-checked build (libgdn_checked.so) on the pooled recurrent rule and the query/key norms: every index
of rows, gates, states, codes and outputs is compared with its buffer's extent before the access. The cases run
in a fresh process; no call may record an index outside (gdn_get_status == GDN_OK), and all must match the
oracle or the formulas."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _recurrent_cases():
    import torch

    import gated_delta_rule_112_b200 as gdn
    from tests import test_recurrent_gpu as t

    assert gdn.lib().gdn_checked_build() == 1, "not the checked library"
    status = gdn.status_block()

    def clean(d, **how):
        o, pool = t.call(d, status=status, **how)
        code = gdn.get_status(status)
        assert code == gdn.OK, (gdn.lib().gdn_status_string(code), status[:16].view(torch.int32).tolist())
        t.check(d, o, pool, **{n: x for n, x in how.items() if n in ("keep", "reset")})

    for i, (lens, *sizes) in enumerate([*t.CASES, *t.STEP]):
        Hk, Hv, dk, dv, *types, channel = sizes if len(sizes) == 7 else (*sizes[:4], t.F, t.BF, sizes[4])
        d = t.make(lens, Hk, Hv, dk, dv, *types, channel, seed=300 + i, spare=0)
        clean(d)
        clean(d, keep=[n // 2 for n in lens], reset=[n % 2 == 0 for n in range(len(lens))])
    for i, (N, *sizes) in enumerate(t.ONE):
        d = t.make([1] * N, *sizes, seed=400 + i, spare=0)
        clean(d, cu=False)
    # slices of one projection's output: strides, the last token's rows at the buffer's end
    for dtype in (t.BF, t.F):
        d = t.make([3, 8], 2, 4, 128, 64, dtype, seed=500, spare=0)
        wide = torch.cat([d[x].flatten(1) for x in "qkv"], 1).cuda()
        q, k, v = (x.unflatten(1, (-1, w)) for x, w in zip(wide.split([256, 256, 256], 1), (128, 128, 64)))
        pool = d["pool"].cuda()
        o = gdn.recurrent_fwd(q, k, v, d["g"].cuda(), d["beta"].cuda(), pool, d["slots"].cuda(), d["cu"].cuda(),
                              status=status)
        assert gdn.get_status(status) == gdn.OK
        t.check(d, o, pool)
    print("checked build: all cases clean")


def _norm_cases():
    import torch

    import gated_delta_rule_112_b200 as gdn
    from tests import test_qk_norm_gpu as t

    assert gdn.lib().gdn_checked_build() == 1, "not the checked library"

    def clean(what):
        code = gdn.get_status()
        assert code == gdn.OK, (what, gdn.lib().gdn_status_string(code))

    for case in range(len(t.CASES)):
        t.test_forward(case)
        clean(("forward", case))
        t.test_codes_are_exact(case)
        clean(("codes", case))
        t.test_backward(case, t.F)
        t.test_backward(case, None)
        clean(("backward", case))
        t.test_from_the_checkpoint(case)
        clean(("from the checkpoint", case))
    for test in (t.test_strided_unaligned_and_in_place, t.test_heads_outermost, t.test_no_tokens_and_one_tensor,
                 t.test_codes_at_the_ends):
        test()
        clean(test.__name__)
    torch.cuda.synchronize()
    print("checked build: all cases clean")


def _run(what):
    from gated_delta_rule_112_b200 import build as gbuild
    env = dict(os.environ, GDN_LIBRARY=gbuild.build(checked=True), PYTHONPATH=ROOT)
    out = subprocess.run([sys.executable, os.path.abspath(__file__), what], cwd=ROOT, env=env, capture_output=True,
                         text=True, timeout=600)
    assert out.returncode == 0, out.stdout[-2000:] + out.stderr[-3000:]
    assert "all cases clean" in out.stdout


@pytest.mark.gpu
def test_checked_build_runs_the_pooled_rule_clean():
    _run("recurrent")


@pytest.mark.gpu
def test_checked_build_runs_the_norms_clean():
    _run("norms")


if __name__ == "__main__":
    sys.path.insert(0, ROOT)
    {"recurrent": _recurrent_cases, "norms": _norm_cases}[sys.argv[1]]()
