"""Rows that are done one by one, because the tensor cores' 0 * v would carry a value that is not finite into rows that do
not see it: how long they take grows with the keys, past the limit of the waits of the warps behind them."""
import math

import pytest
import torch

from tests.test_gpu_prompt_attention import check, cu, draw, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


def attend(B, q, k, v, cq, ck):
    """Causal attention without scratch: nothing is cut, so that a unit goes over all of its keys."""
    (n, Hq, D), (m, Hkv, _) = q.shape, k.shape
    out, lse, st = torch.full_like(q, 7.0), torch.full((n, Hq), 7.0, device="cuda"), B.new_status("cuda")
    work = torch.zeros(B.PROMPT_WORK_WORDS, dtype=torch.int32, device="cuda")
    B._launch("hpc_prompt_attention", q.device, q.data_ptr(), Hq * D, D, k.data_ptr(), Hkv * D, D, v.data_ptr(), Hkv * D, D, n, m,
              cq.data_ptr(), ck.data_ptr(), 1, Hq, Hkv, D, 1, D ** -0.5, out.data_ptr(), lse.data_ptr(), work.data_ptr(),
              None, 0, st.data_ptr())
    return out, lse, int(st.item())


def test_rows_that_outlast_the_waits(B):
    """300 units of 256 queries, the last of which holds a NaN that its first 156 queries do not see. Its rows take longer
    than the waits' 2 s, and its CTA has taken other units by then."""
    n, m, D = 256 * 300, 450_000, 64
    q, k, v = draw(1, n, 1, D), draw(2, m, 1, D), draw(3, m, 1, D)
    cq, ck = cu([n]), cu([m])
    clean, clean_lse, st = attend(B, q, k, v, cq, ck)
    assert st == 0
    v[m - 100, 0, 5] = math.nan
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    out, lse, st = attend(B, q, k, v, cq, ck)
    end.record()
    end.synchronize()
    assert st == 0
    assert start.elapsed_time(end) > 2000  # or the case shows nothing
    last = n - 256
    assert torch.equal(out[:last], clean[:last]) and torch.equal(lse[:last], clean_lse[:last])
    v[m - 100, 0, 5] = 0
    want = reference(q[last:], k, v, D ** -0.5, True)
    check(out[last:n - 100], lse[last:n - 100], [w[:156] for w in want])
    dims = [d for d in range(D) if d != 5]
    check(out[n - 100:, :, dims], lse[n - 100:], [w[156:, :, dims] if w.dim() == 3 else w[156:] for w in want])
    assert torch.isnan(out[n - 100:, :, 5]).all()
