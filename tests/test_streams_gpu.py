"""Calls on a stream that is not the current one, without an output tensor: what
the call allocates belongs to its stream."""

import pytest
import torch

from linear_attention_ssm_step_gb300 import kda, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("prepared", [False, True])
@pytest.mark.parametrize("name", ["decode", "verify", "prefill"])
def test_outputs_are_not_memory_the_current_stream_still_writes(dev, name, prepared):
    """The current stream is busy, then writes into memory that it has given back to its pool."""
    T, shape = (4, (6, 4)) if name == "verify" else (None, (6,))
    w = workloads.decode_inputs(6, 9, seed=31, **({"T": T} if T else {}))
    rest = (w.q, w.k, w.v, w.g_raw, w.beta_logit, w.A_log, w.dt_bias)
    H = w.q.shape[-2]

    def args():
        cu = [torch.tensor([0, 2, 6], dtype=torch.int32, device=dev)] if name == "prefill" else []
        idx = w.state_indices[:2] if name == "prefill" else w.state_indices
        return [x.to(dev) for x in (w.state, idx)] + cu + [x.to(dev) for x in rest]

    one, bound = getattr(kda, "kda_" + name), getattr(kda, "prepare_" + name)
    ref = one(*args())
    side = torch.cuda.Stream()
    for _ in range(5):
        mine = args()
        torch.cuda.synchronize()
        old = [torch.full((*shape, H, 128), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(8)]
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for t in old:
            t.fill_(9)
        del old, t
        out = bound(*mine, stream=side)() if prepared else one(*mine, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
