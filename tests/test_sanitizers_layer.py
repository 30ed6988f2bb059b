"""The decoder-layer calls' host code under the host compiler's AddressSanitizer and UndefinedBehaviorSanitizer: the
refusals of test_boundary_layer, and calls whose arguments pass every check with integers at the ends of their
ranges.  The latter go on to the launch, which fails where there is no device; with one they are skipped (their
pointers are no memory)."""
import glob
import os
import random
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests")


@pytest.fixture(scope="module")
def env():
    from dynamic_scaling_scaled_amd import _build

    sources = _build.sources() + glob.glob(os.path.join(_build.CSRC, "*.h")) + glob.glob(os.path.join(_build.INCLUDE, "*.h"))
    if not os.path.exists(_build.ASAN_LIB) or os.path.getmtime(_build.ASAN_LIB) < max(map(os.path.getmtime, sources)):
        _build.build_host_sanitized()
    runtime = _build.asan_runtime()
    if not runtime:
        pytest.skip("the host compiler's ASan runtime is not installed")
    return dict(os.environ, FP8RT_LIB=_build.ASAN_LIB, LD_PRELOAD=runtime, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0")


def run(env, args):
    r = subprocess.run([sys.executable, *args], cwd=HERE, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    return out


def test_refusals(env):
    out = run(env, ["-m", "pytest", "-q", "-x", "-s", "-p", "no:cacheprovider", "test_boundary_layer.py"])
    assert " passed" in out


SIZES = [1, 2, 15, 16, 17, 64, 128, 256, 4096, 32768, 65535, 2 ** 20, 2 ** 22, 2 ** 23, 2 ** 30, 2 ** 31 - 1, 2 ** 31, 2 ** 40,
         2 ** 62, 2 ** 63 - 16, 2 ** 63 - 1]


def extreme_calls(seed=7, n=1500):
    """Calls with some integers replaced by sizes at the ends of their ranges (run as a script)."""
    sys.path.insert(0, ROOT)
    import dynamic_scaling_scaled_amd as rt
    import test_boundary_layer as t

    rng = random.Random(seed)
    plan = ["tokens", "seqs", "max_new", "width", "ldt", "pages", "heads"]
    sides = [(t.norm, ["rows", "cols", "ldx", "ldr", "ldq", "ldh"]), (t.grad, ["rows", "cols", "lddy", "ldh", "lddx"]),
             (t.append, plan + ["ldk", "hdk", "ldv", "hdv"]),
             (t.attend, plan + ["qh", "ldq", "hdq", "max_kv", "window", "ldy", "hdy"])]
    seen = set()
    for i in range(n):
        for call, names in sides:
            kw = {k: rng.choice(SIZES) for k in rng.sample(names, rng.randint(1, 4))}
            if "width" in kw:
                kw.setdefault("ldt", kw["width"])
            if "heads" in kw and "qh" not in kw and call is t.attend:
                kw["qh"] = kw["heads"] * rng.choice([1, 2, 8, 17])
            seen.add(call(rt, **kw))
    assert t.attend(rt, window=2 ** 63 - 1) == t.attend(rt, window=2 ** 63 - 1, max_new=64, tokens=64) == rt.EHIP
    assert seen == {rt.EINVAL, rt.EALIGN, rt.EUNSUPPORTED, rt.EHIP}, seen  # (no device: no call succeeds)
    print("done")


def test_sizes_at_the_ends_of_their_ranges(env):
    import torch

    if os.path.exists("/dev/kfd") or torch.cuda.is_available():
        pytest.skip("a device is there: calls that pass the checks would run")
    assert "done" in run(env, ["test_sanitizers_layer.py"])


if __name__ == "__main__":
    extreme_calls()
