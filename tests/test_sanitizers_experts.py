"""The host code of the calls of the gated half of a decoder layer under the host compiler's AddressSanitizer and
UndefinedBehaviorSanitizer: the refusals of test_boundary_experts, and calls whose arguments pass every check with
integers at the ends of their ranges.  The latter go on to the launch, which fails where there is no device; with one
they are skipped (their pointers are no memory)."""
import os
import random
import sys

import pytest

from test_sanitizers_layer import ROOT, SIZES, env, run  # noqa: F401 (env: the fixture)


def test_refusals(env):
    out = run(env, ["-m", "pytest", "-q", "-x", "-s", "-p", "no:cacheprovider", "test_boundary_experts.py"])
    assert " passed" in out


def extreme_calls(seed=11, n=1500):
    """Calls with some integers replaced by sizes at the ends of their ranges (run as a script)."""
    sys.path.insert(0, ROOT)
    import dynamic_scaling_scaled_amd as rt
    import test_boundary_experts as t

    rng = random.Random(seed)
    sides = [(t.route, ["tokens", "experts", "ld", "groups", "top", "k"]),
             (t.route_grad, ["tokens", "experts", "ld", "k", "ldd"]),
             (t.gemm, ["rows", "lda", "choices", "experts", "slots", "N", "K", "ldy"]),
             (t.gated, ["rows", "cols", "ldx", "ldq", "ldk"]), (t.gated_grad, ["rows", "cols", "lddz", "ldk", "lddx", "ldz"]),
             (t.combine, ["x_rows", "cols", "ldx", "tokens", "k", "ldr", "ldy"]),
             (t.combine_grad, ["tokens", "cols", "lddy", "x_rows", "ldx", "k", "lddx"])]
    seen = {call.__name__: set() for call, _ in sides}
    for i in range(n):
        for call, names in sides:
            kw = {k: rng.choice(SIZES) for k in rng.sample(names, rng.randint(1, 3))}
            seen[call.__name__].add(call(rt, **kw))
    for name, got in seen.items():  # (no device: no call succeeds)
        assert rt.EHIP in got and rt.EINVAL in got and 0 not in got, (name, got)
    assert t.route(rt, tokens=2 ** 27, k=8) == rt.EHIP
    assert t.gemm(rt, slots=2 ** 20, N=2 ** 12, ldy=2 ** 12, experts=1024) == rt.EHIP
    print("done")


def test_sizes_at_the_ends_of_their_ranges(env):
    import torch

    if os.path.exists("/dev/kfd") or torch.cuda.is_available():
        pytest.skip("a device is there: calls that pass the checks would run")
    assert "done" in run(env, ["test_sanitizers_experts.py"])


if __name__ == "__main__":
    extreme_calls()
