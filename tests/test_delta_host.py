"""CPU tests of the gated delta rule's and the norm-and-turn pass's refusals, all made before
any CUDA call, and of the 64-bit forms the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import kda_prefill_gb300 as kda
from kda_prefill_gb300 import ops
from tests import delta_reference as ref
from tests.test_binding_device_host import _g
from tests.test_ops_host import BASE, LIN_BAD, _bf, _c, lib, lin_args  # noqa: F401

BETA_BAD = {
    "beta_dtype": ({"beta": _c(torch.zeros(1, 96, 4).bfloat16())}, TypeError, "beta must be a float32"),
    "beta_heads": ({"beta": _c(torch.zeros(1, 96, 2))}, ValueError, "beta must be a contiguous"),
    "beta_per_head": ({"beta": _c(torch.zeros(4))}, ValueError, "beta must be a contiguous"),
    "beta_layout": ({"beta": _c(torch.zeros(4, 96).t())}, ValueError, "beta must be a contiguous"),
}


@pytest.mark.parametrize("case", sorted({**LIN_BAD, **BETA_BAD}))
def test_gated_delta_binding_refuses(lib, case):  # noqa: F811
    over, error, message = {**LIN_BAD, **BETA_BAD}[case]
    a = dict(lin_args(), beta=_c(torch.zeros(1, 96, 4)))
    a.update(over)
    args = [a.pop(n) for n in ("q", "k", "v", "log_decay", "beta", "cu_seqlens")]
    with pytest.raises(error, match=message):
        kda.gated_delta_fwd(*args, **a)


def delta_abi(lib, **over):  # noqa: F811
    """kda_gated_delta_fwd with made-up addresses that are right unless `over` says else."""
    cu = over.pop("cu", [0, 37, 96])
    host = torch.tensor(cu, dtype=torch.int32)
    M = 1 << 26
    a = dict(q=BASE, q_st=256, q_sh=128, k=BASE + M, k_st=256, k_sh=128, v=BASE + 2 * M, v_st=512,
             v_sh=128, g=BASE + 3 * M, per_token=1, beta=BASE + 4 * M, cu_dev=BASE + 5 * M,
             host=host.data_ptr(), N=2, T=96, H=4, Hk=2, pool=BASE + 6 * M, stride0=4 * 128 * 128, slots=3,
             idx=BASE + 7 * M, has=BASE + 8 * M, out=BASE + 9 * M, scale=1.0, dtype=0, ws=BASE + 10 * M,
             ws_bytes=1 << 30, stream=None)
    a.update(over)
    rc = lib.kda_gated_delta_fwd(*a.values())
    return rc, lib.kda_last_error().decode()


@pytest.mark.parametrize("over,code,message", [
    (dict(T=-1), -1, "total_tokens"),
    (dict(T=2 ** 31 - 5), -1, "int32 token index"),
    (dict(N=-1), -1, "num_seqs"),
    (dict(H=0), -1, "num_heads"),
    (dict(Hk=3), -1, "does not divide"),
    (dict(dtype=3), -2, "state_dtype"),
    (dict(host=None, cu_dev=None), -1, "both NULL"),
    (dict(cu=[0, 40, 39]), -1, "decreases"),
    (dict(T=95), -1, "expected total_tokens"),
    (dict(k=None), -1, "pointer is NULL"),
    (dict(beta=None), -1, "beta is NULL"),
    (dict(beta=BASE + (4 << 26) + 2), -2, "beta is not"),
    (dict(beta=BASE + (9 << 26) + 16), -1, "out overlaps beta"),
    (dict(beta=BASE + (6 << 26) + 16), -1, "state_cache overlaps beta"),
    (dict(beta=BASE + (10 << 26) + 16), -1, "workspace overlaps beta"),
    (dict(q=BASE + 2), -2, "q and its strides"),
    (dict(v_sh=64), -1, "smaller than a row"),
    (dict(out=BASE + (9 << 26) + 8), -2, "out is not 16-byte"),
    (dict(g=BASE + 2), -2, "log_decay is not"),
    (dict(ws_bytes=8), -5, "workspace of 8 bytes"),
    (dict(ws=None), -5, "workspace of 0 bytes"),
    (dict(ws=BASE + (10 << 26) + 16), -2, "workspace is not"),
    (dict(pool=None), -1, "are required"),
    (dict(slots=1), -1, "num_slots 1"),
    (dict(stride0=4 * 128 * 128 - 1), -1, "smaller than the slot plane"),
    (dict(pool=BASE + (9 << 26)), -1, "state_cache overlaps out"),
])
def test_gated_delta_abi_refuses(lib, over, code, message):  # noqa: F811
    rc, err = delta_abi(lib, **over)
    assert rc == code and message in err, (rc, err)


def test_gated_delta_without_sequences(lib):  # noqa: F811
    assert delta_abi(lib, N=0, T=0, cu=[0])[0] == 0
    assert delta_abi(lib, N=0, T=5, cu=[0])[0] == -1


def test_gated_delta_workspace(lib):  # noqa: F811
    size = kda.gated_delta_workspace_size
    assert size(-1, 1, 1) == 0 and size(1, 1, 0) == 0 and size(5, 0, 3) == 0
    assert size(0, 1, 1) >= 256
    assert size(2000, 3, 4) >= size(1000, 3, 4) >= size(1000, 1, 4) >= size(1000, 1, 1)


def turn_abi(lib, tensors=None, **over):  # noqa: F811
    t = tensors if tensors is not None else [((BASE, BASE + (1 << 24), 512, 128, 512, 128, 4), BASE + (5 << 24), 0)]
    arr = (ops._NormRopeTensor * 2)(*[ops._NormRopeTensor(*x) for x in t])
    a = dict(t=arr, n=len(t), eps=1e-6, pos=BASE + (2 << 24), pos_bytes=4, freq=BASE + (3 << 24), T=96, D=128,
             rot=128, layout=0, factor=1.0, dtype=1, stream=None)
    a.update(over)
    rc = lib.kda_qk_norm_rope(*a.values())
    return rc, lib.kda_last_error().decode()


ROW = (BASE, BASE + (1 << 24), 512, 128, 512, 128, 4)


@pytest.mark.parametrize("tensors,over,code,message", [
    (None, dict(T=-1), -1, "total_tokens"),
    (None, dict(n=0), -1, "kda_qk_norm_rope takes 1 or 2 tensors"),
    (None, dict(n=3), -1, "1 or 2 tensors"),
    (None, dict(t=None), -1, "1 or 2 tensors"),
    (None, dict(eps=-1.0), -1, "eps"),
    (None, dict(eps=float("nan")), -1, "eps"),
    (None, dict(D=0), -2, "head_dim"),
    (None, dict(D=1025), -2, "head_dim"),
    (None, dict(rot=127), -1, "rot_dim"),
    (None, dict(layout=2), -2, "layout"),
    (None, dict(dtype=5), -2, "dtype"),
    (None, dict(pos_bytes=2), -2, "positions of 2 bytes"),
    (None, dict(pos=None), -1, "are required"),
    (None, dict(pos=BASE + (1 << 24)), -1, "overlaps the positions"),
    ([(ROW, BASE + 2, 0)], {}, -2, "weight 0 is not"),
    ([(ROW, BASE + (5 << 24), -128)], {}, -1, "weight_stride_h"),
    ([(ROW, BASE + (1 << 24) + 64, 0)], {}, -1, "overlaps a weight"),
    ([(ROW, None, 0), ((BASE + (6 << 24), BASE + (6 << 24), 512, 128, 512, 128, 4), BASE + (1 << 24) - 1024, 128)], {}, -1,
     "overlaps a weight"),
    ([((BASE, BASE + 256, 512, 128, 512, 128, 4), None, 0)], {}, -1, "overlaps its in"),
    ([((BASE, BASE, 512, 128, 512, 128, -1), None, 0)], {}, -1, "num_heads"),
])
def test_qk_norm_rope_abi_refuses(lib, tensors, over, code, message):  # noqa: F811
    rc, err = turn_abi(lib, tensors, **over)
    assert rc == code and message in err, (rc, err)


def test_qk_norm_rope_without_work(lib):  # noqa: F811
    assert turn_abi(lib, T=0)[0] == 0
    assert turn_abi(lib, [((BASE, BASE, 512, 128, 512, 128, 0), None, 0)])[0] == 0


def test_qk_norm_rope_binding_refuses(lib):  # noqa: F811
    q, k = _bf(1, 8, 2, 64), _bf(1, 8, 1, 64)
    w = _c(torch.ones(64))
    pos, f = _c(torch.zeros(8, dtype=torch.int32)), _c(torch.ones(32, dtype=torch.float64))
    for args, kw, error, message in [
        ((q, k, w, w, pos, f), dict(layout="odd"), ValueError, "layout"),
        ((_c(torch.zeros(1, 8, 2, 64).double()), k, w, w, pos, f), {}, TypeError, "not supported"),
        ((q, _bf(1, 8, 2, 32), w, w, pos, f), {}, ValueError, "q's T and D"),
        ((q, None, w, None, pos, f), dict(k_out=k), ValueError, "without k"),
        ((q, k, w, w, pos[:7], f), {}, ValueError, "8 entries"),
        ((q, k, w, w, pos, f.float()), {}, TypeError, "float64"),
    ]:
        with pytest.raises(error, match=message):
            kda.qk_norm_rope(*args, **kw)


def test_weights_are_checked(lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(ops, "_on_current_device", lambda at: None)
    q, k = _bf(1, 8, 2, 64), _bf(1, 8, 1, 64)
    w = _c(torch.ones(64))
    pos, f = _c(torch.zeros(8, dtype=torch.int32)), _c(torch.ones(32, dtype=torch.float64))
    for qw, kw, error, message in [
        (w.bfloat16(), w, TypeError, "q_weight must be a float32"),
        (w, w.double(), TypeError, "k_weight must be a float32"),
        (_c(torch.ones(63)), w, ValueError, "q_weight must be a contiguous"),
        (_c(torch.ones(3, 64)), w, ValueError, "q_weight must be a contiguous"),
        (w, _c(torch.ones(2, 64)), ValueError, "k_weight must be a contiguous"),
        (_c(torch.ones(64, 2).t()), w, ValueError, "q_weight must be a contiguous"),
    ]:
        with pytest.raises(error, match=message):
            kda.qk_norm_rope(q, k, qw, kw, pos, f)
    with pytest.raises(ValueError, match="without k"):
        kda.qk_norm_rope(q, None, w, w, pos, f)


def test_tensors_of_another_gpu_are_refused(lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    bf = lambda *s: _g(torch.zeros(*s, dtype=torch.bfloat16))  # noqa: E731
    with pytest.raises(ValueError, match="on cuda:1, and the current device is cuda:0"):
        kda.gated_delta_fwd(bf(1, 96, 2, 128), bf(1, 96, 2, 128), bf(1, 96, 4, 128), _g(torch.zeros(4)),
                            _g(torch.zeros(1, 96, 4)), _g(torch.tensor([0, 37, 96], dtype=torch.int32)),
                            state_cache=_g(torch.zeros(3, 4, 128, 128)),
                            state_indices=_g(torch.zeros(2, dtype=torch.int32)),
                            has_initial_state=_g(torch.zeros(2, dtype=torch.bool)), out=bf(1, 96, 4, 128),
                            cu_seqlens_cpu=torch.tensor([0, 37, 96], dtype=torch.int32))
    with pytest.raises(ValueError, match="on cuda:1, and the current device is cuda:0"):
        kda.qk_norm_rope(bf(1, 8, 2, 64), bf(1, 8, 1, 64), None, None, _g(torch.zeros(8, dtype=torch.int32)),
                         _g(torch.ones(32, dtype=torch.float64)))


def test_struct_matches_the_header(lib):  # noqa: F811
    assert ctypes.sizeof(ops._RopeTensor) == 56 and ctypes.sizeof(ops._NormRopeTensor) == 72


def test_references_agree_with_closed_forms():
    """One key in all tokens, beta = 1: the state gives v for it, whatever was there."""
    k = torch.zeros(3, 1, 2)
    k[..., 0] = 1000.0
    v = torch.tensor([[[1.0, 2.0]], [[3.0, 4.0]], [[5.0, 7.0]]])
    o, S, emag, fmag = ref.gated_delta(k, k, v, torch.zeros(1), torch.ones(3, 1), [3],
                                       torch.full((1, 1, 2, 2), 8.0), [1], 2.0)
    assert o[:, 0].tolist() == [pytest.approx(x) for x in ([2.0, 4.0], [6.0, 8.0], [10.0, 14.0])]
    assert S[0, 0].tolist() == [pytest.approx([5.0, 8.0]), pytest.approx([7.0, 8.0])]
    assert fmag[0, 0].tolist() == pytest.approx([128 ** 0.5 + 7 + 2 + 2, 128 ** 0.5 + 6 + 2 + 3])
    # beta = 0: the states decay
    o, S, *_ = ref.gated_delta(k, k, v, torch.log(torch.tensor([0.5])), torch.zeros(3, 1), [3],
                               torch.full((1, 1, 2, 2), 8.0), [1], 1.0)
    assert S[0, 0].tolist() == [pytest.approx([1.0, 1.0])] * 2 and o[2, 0].tolist() == pytest.approx([1.0, 1.0])
    # two sequences, out of order of their lengths
    a = ref.gated_delta(k, k, v, torch.zeros(1), torch.ones(3, 1), [1, 2], torch.zeros(2, 1, 2, 2), [0, 0], 1.0)
    assert a[1][0, 0, :, 0].tolist() == pytest.approx([1.0, 2.0]) and a[1][1, 0, :, 0].tolist() == pytest.approx([5.0, 7.0])
    x = torch.tensor([[[3.0, 4.0, 0.0]]])
    y = ref.qk_norm_rope(x, torch.tensor([1.0, 2.0, 3.0]), torch.tensor([1]), torch.tensor([math.pi / 2]), "half", 1.0, 0.0)
    r = math.sqrt(25 / 3)
    assert y[0, 0].tolist() == pytest.approx([-8 / r, 3 / r, 0.0])
