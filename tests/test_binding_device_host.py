"""CPU tests that the binding refuses tensors of a GPU that is not the current one.  The
library runs on the current device, where their addresses mean other memory or none; the
tensors here only say that they are on GPU 1, and every call stops before the library."""
import pytest
import torch

import kda_prefill_gb300 as kda
from kda_prefill_gb300 import workloads as wl
from tests.test_ops_host import lib  # noqa: F401  (a fixture)


class _OnGpu1(torch.Tensor):
    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return 1


def _g(x):
    return x.as_subclass(_OnGpu1)


def _bf(*shape):
    return _g(torch.zeros(*shape, dtype=torch.bfloat16))


def lin_attn():
    kda.lin_attn_fwd(_bf(1, 96, 2, 128), _bf(1, 96, 2, 128), _bf(1, 96, 4, 128), _g(torch.zeros(4)),
                     _g(torch.tensor([0, 37, 96], dtype=torch.int32)), state_cache=_g(torch.zeros(3, 4, 128, 128)),
                     state_indices=_g(torch.zeros(2, dtype=torch.int32)),
                     has_initial_state=_g(torch.zeros(2, dtype=torch.bool)), out=_bf(1, 96, 4, 128),
                     cu_seqlens_cpu=torch.tensor([0, 37, 96], dtype=torch.int32))


def rope():
    kda.rope(_bf(1, 8, 2, 64), _bf(1, 8, 1, 64), _g(torch.zeros(8, dtype=torch.int32)),
             _g(torch.ones(32, dtype=torch.float64)))


def gated_norm():
    kda.gated_norm(_bf(1, 8, 2, 64), _g(torch.ones(64)), out=_bf(1, 8, 2, 64))


def _chunk(dense):
    w = wl.make_workload("binding_device", [37, 0, 59], 2, num_slots=5, seed=3)
    S, stride0 = w.pool_storage.shape
    pool = w.pool_storage.as_strided((S, 2, 128, 128), (stride0, 128 * 128, 128, 1))
    a = [_g(x) for x in (w.q, w.k, w.v, w.g_raw, w.beta_raw, w.cu_seqlens)]
    kw = dict(out=_g(torch.empty_like(w.v)), cu_seqlens_cpu=w.cu_seqlens)
    if dense:
        kda.chunk_fwd_dense(*a, final_state=_g(torch.zeros(3, 2, 128, 128)), **kw)
    else:
        kda.chunk_fwd(*a, state_cache=_g(pool), state_indices=_g(w.state_indices),
                      has_initial_state=_g(w.has_initial_state), **kw)


CALLS = {"lin_attn_fwd": lin_attn, "rope": rope, "gated_norm": gated_norm,
         "chunk_fwd": lambda: _chunk(False), "chunk_fwd_dense": lambda: _chunk(True)}


@pytest.mark.parametrize("call", sorted(CALLS))
def test_tensors_of_another_gpu_are_refused(lib, monkeypatch, call):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="on cuda:1, and the current device is cuda:0"):
        CALLS[call]()
