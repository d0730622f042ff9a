"""tree_decode when its waits run out: the call ends with a status, and the next one is right."""

import numpy as np
import pytest

import top_sparse_decode_topk_b200 as tsd
from tests.test_gpu_speculative import i32, status
from tests.test_gpu_tree_wide import filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("n", [6, 80])
@pytest.mark.parametrize("qt,ot", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_waits_that_run_out_are_reported(qt, ot, n, page, monkeypatch):
    import torch
    status()
    dts = {"bf16": torch.bfloat16, "f32": torch.float32}
    rng = np.random.default_rng(n)
    lens = [n + int(x) for x in rng.integers(0, 9000, 12)]
    cache, table = filled(lens, 4, page, n)
    q = torch.randn(12 * n, 16, 128, device="cuda").to(dts[qt])
    qs = tsd.Queries(q, i32(np.arange(13) * n), n)
    call = lambda st: tsd.tree_decode(cache, qs, None, out_dtype=dts[ot], status=st)
    st = i32([0])
    want = call(st)
    assert int(st) == 0
    monkeypatch.setenv("TSD_TREE_WAIT_TRIES", "1")   # a microsecond: less than any tile takes to arrive
    call(st)
    assert int(st) == tsd.DEV_TIMEOUT
    monkeypatch.delenv("TSD_TREE_WAIT_TRIES")
    st.zero_()
    got = call(st)
    assert int(st) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
    assert status() == 0
