"""Plans of different sizes at once (fmha_page_plan): what one call sets must not undo another's."""
import threading

import pytest
import torch

from tests import page_util as pu
from tests import test_page_plan_gpu as tp
from tests.test_page_plan_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def case(B):
    return tp.make([(i * 13) % 40 for i in range(B)], [i % 3 for i in range(B)], 16, B, seed=B)


def want(c):
    return pu.plan(c["seqlen"], c["n_new"], [list(r) for r in c["table"]], list(c["free_list"]), c["n_free"], c["page"], c["rows"], c["entry"])


def test_calls_of_two_threads(fm):  # noqa: F811
    """Each on a stream of its own, one with most sequences, one with as few as need the larger limit."""
    codes, barrier, calls = [], threading.Barrier(2), 3000
    plans = []
    for B in (8192, 2100):
        c = case(B)                                      # no request gives pages back: a call changes nothing that the next one reads
        a, kw = tp.on_gpu(c, False)
        out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (c["rows"], c["rows"], B + 1, B)]
        p = [a["seqlen"], a["n_new"], kw["batch_idx"], a["table"], a["free_list"], a["n_free"], kw["n_free_out"], *out]
        plans.append((c, p, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(c, p, stream):
        f, args = fm.lib().fmha_page_plan, [t.data_ptr() for t in p]
        args += [len(c["seqlen"]), c["rows"], *p[3].shape, p[4].shape[0], 16, stream.cuda_stream]
        barrier.wait()
        codes.append({f(*args) for _ in range(calls)})   # the C call: without the interpreter's lock

    threads = [threading.Thread(target=work, args=x) for x in plans]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}, {0}] and fm.device_status(reset=True) == 0
    for c, p, _ in plans:
        assert [x.tolist() for x in p[7:]] == list(want(c))[:4]


def test_a_graph_of_a_large_call_beside_a_smaller_one(fm):  # noqa: F811
    c, d = case(8192), case(2100)
    (a, kw), (b, kwb) = tp.on_gpu(c, False), tp.on_gpu(d, False)
    keep = {k: v.clone() for k, v in a.items()}
    fm.page_plan(**a, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fm.page_plan(**a, **kw)
        fm.page_plan(**b, **kwb)
    fm.page_plan(**tp.on_gpu(d, False)[0], **kwb)
    for k, v in keep.items():
        a[k].copy_(v)
    g.replay()
    torch.cuda.synchronize()
    assert [x.tolist() for x in out] == list(want(c))[:4] and fm.device_status(reset=True) == 0
