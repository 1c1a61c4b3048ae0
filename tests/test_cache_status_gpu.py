"""fmha_device_status: what it says of work on streams that do not wait for the
default one, and after errors of several operators."""
import pytest
import torch

from tests import test_tree_gpu as tt
from tests.test_tree_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_status_covers_work_on_every_stream(fm):  # noqa: F811
    """A length outside its bounds, met by a kernel that has not begun yet: the call synchronises the device."""
    c = tt.make("bf16", 4, 8, 2, 200, [100, 50], seed=91)
    d, (o, lse) = tt.on_gpu(c), tt.outputs(c)
    fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse)
    d["args"][5] = torch.tensor([201, 50], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse)
    assert not side.query()
    assert fm.device_status() == fm.ERR_INVALID_ARG and side.query()
    assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG    # the call before left it
    assert fm.device_status() == 0


def bad_call(fm, op):  # noqa: F811
    """A call of `op` with a length past its entry's rows, which the kernel clamps and reports."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    kc, vc, long = bf(1, 8, 2, 128), bf(1, 8, 2, 128), i32(9)
    if op == "gen":
        fm.gen_fwd(bf(1, 4, 128), kc, vc, long)
    elif op == "tree":
        fm.tree_fwd(bf(1, 3, 4, 128), kc, vc, bf(1, 3, 2, 128), bf(1, 3, 2, 128), long)
    elif op == "commit":
        fm.tree_commit(kc, vc, bf(1, 3, 2, 128), bf(1, 3, 2, 128), long, i32(0)[None], i32(1))
    elif op == "weights":
        fm.cache_weights(bf(1, 3, 4, 128), kc, torch.zeros((1, 4, 3), device="cuda"), long)
    else:
        fm.cache_evict(kc, vc, torch.zeros((1, 2, 8), device="cuda"), long, 4)


def test_status_of_every_operator(fm):  # noqa: F811
    ops = ("gen", "tree", "commit", "weights", "evict")
    assert fm.device_status(reset=True) == 0
    for op in ops:
        bad_call(fm, op)
        assert fm.device_status() == fm.ERR_INVALID_ARG, op
        assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG and fm.device_status() == 0, op
    for op in ops:
        bad_call(fm, op)
    assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG and fm.device_status() == 0    # all of them cleared


def test_status_takes_no_round_trip_per_operator(fm):  # noqa: F811
    """One launch and one copy: at most four round trips' time, where a copy for each file's word took six."""
    import time
    x = torch.zeros(1, device="cuda")

    def best(f):
        t = []
        for _ in range(10):
            a = time.perf_counter()
            for _ in range(50):
                f()
            t.append(time.perf_counter() - a)
        return min(t)
    assert best(fm.device_status) < 4 * best(x.item)
