"""What the binding of the logits operators passes on and refuses, without a GPU: the library, the
tensors' checks and the streams are stood in for."""
import types

import pytest

import rollout_logprob_consistency_gb300 as tim
from rollout_logprob_consistency_gb300 import binding

torch = pytest.importorskip("torch")


@pytest.fixture
def passed(monkeypatch):
    """The tim_sample_params of the calls of tim.sample on CPU tensors."""
    got = []

    class Lib:
        @staticmethod
        def tim_sample(*args):
            got.append(args[6]._obj)
            return 0

    monkeypatch.setattr(binding, "lib", lambda: Lib)
    monkeypatch.setattr(binding, "_logits_args", lambda t, name: (*t.shape, 0, t.shape[1]))
    monkeypatch.setattr(binding, "_vector", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(binding, "_run", lambda dev, stream, call: call(None))
    return got


def _sample(**kw):
    z, u = torch.zeros(2, 8), torch.zeros(2)
    ws = types.SimpleNamespace(ptr=0, nbytes=1024, buf=z)
    tim.sample(z, u, out=(u, u, u, u), workspace=ws, check=False, **kw)


@pytest.mark.parametrize("top_k,want", [
    (0, 0), (-1, 0), (5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
    (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63 - 1, 2 ** 31 - 1), (-2 ** 31 - 3, 0), (-2 ** 32 + 7, 0)])
def test_top_k_beyond_32_bits_is_off_not_another_number(passed, top_k, want):
    """Any number from the vocabulary's size up means all tokens, any below 1 too."""
    _sample(top_k=top_k)
    assert max(passed[0].top_k, 0) == want


def test_a_stream_of_another_device_is_refused():
    """Its kernels would read the tensors from a device that need not see them."""
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=64)
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        binding._run(torch.device("cuda", 0), stream, lambda sp: pytest.fail("launched"))


@pytest.mark.parametrize("op", ["sample", "distill", "distill_grad"])
def test_a_workspace_of_another_device_is_refused(monkeypatch, op):
    """A kernel writes its status there."""
    monkeypatch.setattr(binding, "lib", lambda: pytest.fail("launched"))
    monkeypatch.setattr(binding, "_logits_args", lambda t, name: (*t.shape, 0, t.shape[1]))
    monkeypatch.setattr(binding, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(binding, "_run", lambda dev, stream, call: call(None))
    ws = types.SimpleNamespace(ptr=0, nbytes=1024, buf=torch.zeros(1, device="meta"))
    z, u = torch.zeros(2, 8), torch.zeros(2)
    ids, lp, saved = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2, 8)
    with pytest.raises(ValueError, match="workspace must be on cpu"):
        if op == "sample":
            tim.sample(z, u, out=(u, u, u, u), workspace=ws, check=False)
        elif op == "distill":
            tim.distill(z, ids, lp, out=(u, u, saved), workspace=ws, check=False)
        else:
            tim.distill_grad(z, ids, lp, u, out_dlogits=torch.zeros(2, 8), workspace=ws, check=False)
