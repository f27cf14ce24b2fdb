"""The smoke call reaches both kernels of the attention over a paged cache in 8 bits."""

import pytest
import torch

from linear_attention_ssm_step_gb300 import kda

pytestmark = pytest.mark.gpu


def test_smoke_attends_with_few_rows_and_with_chunks(monkeypatch):
    """Requests with up to 32 rows a key-value head on average go to the kernel for few rows, others to the one for chunks."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    call, rows = kda.kda_paged_attention_fp8, []

    def recorded(q, k_codes, *rest, **kw):
        requests = rest[5].numel()  # kv_len
        rows.append(-(-q.shape[0] // requests) * (q.shape[1] // k_codes.shape[2]))
        return call(q, k_codes, *rest, **kw)

    monkeypatch.setattr(kda, "kda_paged_attention_fp8", recorded)
    __graft_entry__.smoke()
    assert min(rows) <= 4 and any(4 < r <= 32 for r in rows) and max(rows) > 32
