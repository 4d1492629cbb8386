"""CPU tests of the operators beside the KDA forward: the binding's and the C
ABI's refusals, all made before any CUDA call, and the rotary frequencies."""
import ctypes
import math

import pytest
import torch

import kda_prefill_gb300 as kda
from kda_prefill_gb300 import build as kbuild
from kda_prefill_gb300 import ops


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


class _AsCuda(torch.Tensor):
    """A CPU tensor that passes the binding's `is_cuda` test."""

    @property
    def is_cuda(self):
        return True


def _c(x):
    return x.as_subclass(_AsCuda)


def _bf(*shape):
    return _c(torch.zeros(*shape, dtype=torch.bfloat16))


def lin_args():
    return dict(q=_bf(1, 96, 2, 128), k=_bf(1, 96, 2, 128), v=_bf(1, 96, 4, 128),
                log_decay=_c(torch.zeros(4)), cu_seqlens=_c(torch.tensor([0, 37, 96], dtype=torch.int32)),
                state_cache=_c(torch.zeros(3, 4, 128, 128)),
                state_indices=_c(torch.zeros(2, dtype=torch.int32)),
                has_initial_state=_c(torch.zeros(2, dtype=torch.bool)), out=_bf(1, 96, 4, 128),
                cu_seqlens_cpu=torch.tensor([0, 37, 96]))


LIN_BAD = {
    "q_dtype": ({"q": _c(torch.zeros(1, 96, 2, 128))}, TypeError, "q must be torch.bfloat16"),
    "batch": ({"q": _bf(2, 48, 2, 128)}, ValueError, "batch dim 1"),
    "head_size": ({"q": _bf(1, 96, 2, 64)}, ValueError, "must be \\[1, T, Hqk, 128\\]"),
    "k_heads": ({"k": _bf(1, 96, 4, 128)}, ValueError, "must be \\[1, T, Hqk, 128\\]"),
    "groups": ({"q": _bf(1, 96, 3, 128), "k": _bf(1, 96, 3, 128)}, ValueError, "not a multiple of 3"),
    "inner_stride": ({"v": _bf(1, 96, 128, 4).transpose(2, 3)}, ValueError, "dense in its last"),
    "decay_dtype": ({"log_decay": _c(torch.zeros(4).half())}, TypeError, "float32"),
    "decay_shape": ({"log_decay": _c(torch.zeros(5))}, ValueError, "contiguous \\[H\\]"),
    "decay_layout": ({"log_decay": _c(torch.zeros(4, 96).t())}, ValueError, "contiguous \\[H\\]"),
    "bounds_dtype": ({"cu_seqlens": _c(torch.tensor([0, 37, 96]))}, TypeError, "int32"),
    "host_bounds": ({"cu_seqlens_cpu": torch.tensor([0, 96])}, ValueError, "has 2 bounds"),
    "out_shape": ({"out": _bf(1, 96, 2, 128)}, ValueError, "shape of v"),
    "out_layout": ({"out": _bf(1, 4, 96, 128).transpose(1, 2)}, ValueError, "contiguous"),
    "pool_dtype": ({"state_cache": _c(torch.zeros(3, 4, 128, 128).double())}, TypeError, "not supported"),
    "pool_shape": ({"state_cache": _c(torch.zeros(3, 2, 128, 128))}, ValueError, "slots, H, 128, 128"),
    "pool_plane": ({"state_cache": _c(torch.zeros(3, 4, 128, 256))[..., :128]}, ValueError, "may pad"),
    "indices": ({"state_indices": _c(torch.zeros(3, dtype=torch.int32))}, ValueError, "2 entries"),
    "flags": ({"has_initial_state": _c(torch.zeros(2))}, TypeError, "bool/uint8"),
    "workspace": ({"workspace": torch.zeros(16, dtype=torch.uint8)}, ValueError, "too small"),
}


@pytest.mark.parametrize("case", sorted(LIN_BAD))
def test_lin_attn_binding_refuses(lib, case):
    over, error, message = LIN_BAD[case]
    a = dict(lin_args(), **over)
    with pytest.raises(error, match=message):
        kda.lin_attn_fwd(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("log_decay"), a.pop("cu_seqlens"), **a)


BASE = 1 << 40  # addresses are checked, never touched


def lin_abi(lib, **over):
    """kda_lin_attn_fwd with made-up addresses that are right unless `over` says else."""
    cu = over.pop("cu", [0, 37, 96])
    host = torch.tensor(cu, dtype=torch.int32)
    M = 1 << 24
    a = dict(q=BASE, q_st=256, q_sh=128, k=BASE + M, k_st=256, k_sh=128, v=BASE + 2 * M, v_st=512,
             v_sh=128, g=BASE + 3 * M, per_token=1, cu_dev=BASE + 4 * M, host=host.data_ptr(), N=2,
             T=96, H=4, Hk=2, pool=BASE + 5 * M, stride0=4 * 128 * 128, slots=3, idx=BASE + 6 * M,
             has=BASE + 7 * M, out=BASE + 8 * M, scale=1.0, dtype=0, ws=BASE + 9 * M, ws_bytes=1 << 24,
             stream=None)
    a.update(over)
    rc = lib.kda_lin_attn_fwd(*a.values())
    return rc, lib.kda_last_error().decode()


@pytest.mark.parametrize("over,code,message", [
    (dict(T=-1), -1, "total_tokens"),
    (dict(T=2 ** 31 - 5), -1, "int32 token index"),
    (dict(N=-1), -1, "num_seqs"),
    (dict(H=0), -1, "num_heads"),
    (dict(Hk=3), -1, "does not divide"),
    (dict(Hk=0), -1, "does not divide"),
    (dict(dtype=3), -2, "state_dtype"),
    (dict(host=None, cu_dev=None), -1, "both NULL"),
    (dict(cu=[0, 40, 39]), -1, "decreases"),
    (dict(cu=[1, 37, 96]), -1, "expected 0"),
    (dict(T=95), -1, "expected total_tokens"),
    (dict(q=None), -1, "pointer is NULL"),
    (dict(g=None), -1, "pointer is NULL"),
    (dict(q=BASE + 2), -2, "q and its strides"),
    (dict(k_st=260), -2, "k and its strides"),
    (dict(v_sh=64), -1, "smaller than a row"),
    (dict(v_st=-512), -1, "smaller than a row"),
    (dict(q_st=1 << 57), -1, "out of range"),
    (dict(out=BASE + 8), -2, "out is not 16-byte"),
    (dict(out=BASE + 256), -1, "out overlaps q"),
    (dict(g=BASE + 2), -2, "log_decay is not"),
    (dict(ws_bytes=8), -5, "workspace of 8 bytes"),
    (dict(ws=None), -5, "workspace of 0 bytes"),
    (dict(ws=BASE + (9 << 24) + 16), -2, "workspace is not"),
    (dict(ws=BASE + (5 << 24)), -1, "overlaps workspace"),
    (dict(ws=BASE + (2 << 24)), -1, "workspace overlaps v"),
    (dict(pool=None), -1, "are required"),
    (dict(slots=1), -1, "num_slots 1"),
    (dict(stride0=4 * 128 * 128 - 1), -1, "smaller than the slot plane"),
    (dict(stride0=1 << 60), -1, "out of range"),
    (dict(stride0=4 * 128 * 128 + 2), -2, "slot stride"),
    (dict(pool=BASE + (8 << 24)), -1, "state_cache overlaps out"),
])
def test_lin_attn_abi_refuses(lib, over, code, message):
    rc, err = lin_abi(lib, **over)
    assert rc == code and message in err, (rc, err)


def test_lin_attn_without_sequences(lib):
    assert lin_abi(lib, N=0, T=0, cu=[0])[0] == 0
    assert lin_abi(lib, N=0, T=5, cu=[0])[0] == -1


def test_lin_attn_workspace(lib):
    assert kda.lin_attn_workspace_size(-1, 1, 1) == 0 and kda.lin_attn_workspace_size(1, 1, 0) == 0
    assert kda.lin_attn_workspace_size(5, 0, 3) == 0
    assert kda.lin_attn_workspace_size(0, 1, 1) >= 256


def rope_abi(lib, tensors=None, **over):
    t = tensors if tensors is not None else [(BASE, BASE + (1 << 24), 512, 128, 512, 128, 4)]
    arr = (ops._RopeTensor * 2)(*[ops._RopeTensor(*x) for x in t])
    a = dict(t=arr, n=len(t), pos=BASE + (2 << 24), pos_bytes=4, freq=BASE + (3 << 24), T=96, D=128,
             rot=128, layout=0, factor=1.0, inverse=0, dtype=1, stream=None)
    a.update(over)
    rc = lib.kda_rope(*a.values())
    return rc, lib.kda_last_error().decode()


@pytest.mark.parametrize("tensors,over,code,message", [
    (None, dict(T=-1), -1, "total_tokens"),
    (None, dict(n=0), -1, "1 or 2 tensors"),
    (None, dict(n=3), -1, "1 or 2 tensors"),
    (None, dict(t=None), -1, "1 or 2 tensors"),
    (None, dict(D=0), -2, "head_dim"),
    (None, dict(D=1025), -2, "head_dim"),
    (None, dict(rot=127), -1, "rot_dim"),
    (None, dict(rot=130), -1, "rot_dim"),
    (None, dict(rot=-2), -1, "rot_dim"),
    (None, dict(layout=2), -2, "layout"),
    (None, dict(dtype=5), -2, "dtype"),
    (None, dict(pos_bytes=2), -2, "positions of 2 bytes"),
    (None, dict(pos=None), -1, "are required"),
    (None, dict(freq=None), -1, "are required"),
    (None, dict(freq=BASE + (3 << 24) + 4), -2, "aligned to its type"),
    (None, dict(pos=BASE + (1 << 24)), -1, "overlaps the positions"),
    ([(None, BASE, 512, 128, 512, 128, 4)], {}, -1, "NULL pointer"),
    ([(BASE + 1, BASE + 9, 512, 128, 512, 128, 4)], {}, -2, "2-byte aligned"),
    ([(BASE, BASE + (1 << 24), 512, 127, 512, 128, 4)], {}, -1, "smaller than a row"),
    ([(BASE, BASE + (1 << 24), 512, 128, 130, 128, 4)], {}, -1, "make its rows overlap"),
    ([(BASE, BASE + 256, 512, 128, 512, 128, 4)], {}, -1, "overlaps its in"),
    ([(BASE, BASE, 512, 128, 1024, 128, 4)], {}, -1, "overlaps its in"),
    ([(BASE, BASE, 512, 128, 512, 128, -1)], {}, -1, "num_heads"),
])
def test_rope_abi_refuses(lib, tensors, over, code, message):
    rc, err = rope_abi(lib, tensors, **over)
    assert rc == code and message in err, (rc, err)


def norm_abi(lib, **over):
    a = dict(x=BASE, x_st=512, x_sh=128, gate=BASE + (1 << 24), g_st=512, g_sh=128, w=BASE + (2 << 24),
             out=BASE + (3 << 24), o_st=512, o_sh=128, T=96, H=4, D=128, eps=1e-6, act=1, dtype=1,
             stream=None)
    a.update(over)
    rc = lib.kda_gated_norm(*a.values())
    return rc, lib.kda_last_error().decode()


@pytest.mark.parametrize("over,code,message", [
    (dict(T=-1), -1, "total_tokens"),
    (dict(H=-1), -1, "num_heads"),
    (dict(D=0), -2, "head_dim"),
    (dict(D=8193), -2, "head_dim"),
    (dict(eps=-1.0), -1, "eps"),
    (dict(eps=float("nan")), -1, "eps"),
    (dict(act=3), -2, "activation"),
    (dict(dtype=-1), -2, "dtype"),
    (dict(x=None), -1, "NULL"),
    (dict(out=None), -1, "NULL"),
    (dict(gate=BASE + 1), -2, "aligned"),
    (dict(w=BASE + 2), -2, "aligned"),
    (dict(x_st=100), -1, "smaller than a row"),
    (dict(g_sh=100), -1, "smaller than a row"),
    (dict(o_st=200), -1, "make its rows overlap"),
    (dict(out=BASE + 256), -1, "out overlaps x"),
    (dict(out=BASE, o_st=1024), -1, "out overlaps x"),
    (dict(out=BASE + (1 << 24)), -1, "out overlaps gate"),
    (dict(out=BASE + (2 << 24)), -1, "out overlaps weight"),
])
def test_gated_norm_abi_refuses(lib, over, code, message):
    rc, err = norm_abi(lib, **over)
    assert rc == code and message in err, (rc, err)


def test_rope_binding_refuses(lib):
    q, k = _bf(1, 8, 2, 64), _bf(1, 8, 1, 64)
    pos, f = _c(torch.zeros(8, dtype=torch.int32)), _c(torch.ones(32, dtype=torch.float64))
    for args, kw, error, message in [
        ((q, k, pos, f), dict(layout="odd"), ValueError, "layout"),
        ((_c(torch.zeros(1, 8, 2, 64).double()), k, pos, f), {}, TypeError, "not supported"),
        ((q, _c(torch.zeros(1, 8, 2, 64)), pos, f), {}, TypeError, "k must be"),
        ((q, _bf(1, 8, 2, 32), pos, f), {}, ValueError, "q's T and D"),
        ((q, k, pos, f), dict(q_out=_bf(1, 8, 3, 64)), ValueError, "q's T and D"),
        ((q, None, pos, f), dict(k_out=k), ValueError, "without k"),
        ((q, k, pos.float(), f), {}, TypeError, "int32 or int64"),
        ((q, k, pos[:7], f), {}, ValueError, "8 entries"),
        ((q, k, pos, f.float()), {}, TypeError, "float64"),
        ((q, k, pos, _c(torch.ones(33, dtype=torch.float64))), {}, ValueError, "at most D / 2"),
    ]:
        with pytest.raises(error, match=message):
            kda.rope(*args, **kw)


def test_gated_norm_binding_refuses(lib):
    x, w = _bf(1, 8, 2, 64), _c(torch.ones(64))
    for args, kw, error, message in [
        ((x, w), dict(activation="relu"), ValueError, "activation"),
        ((_c(torch.zeros(1, 8, 2, 64).double()), w), {}, TypeError, "not supported"),
        ((x, w), dict(out=_bf(1, 8, 2, 32)), ValueError, "shape of x"),
        ((x, w), dict(out=_bf(1, 8, 2, 64), gate=_bf(1, 8, 1, 64)), ValueError, "shape of x"),
        ((x, w), dict(out=_bf(1, 8, 2, 64), gate=_c(torch.zeros(1, 8, 2, 64))), TypeError, "gate must be"),
        ((x, _c(torch.ones(63))), dict(out=_bf(1, 8, 2, 64)), ValueError, "64 values"),
        ((x, w.bfloat16()), dict(out=_bf(1, 8, 2, 64)), TypeError, "float32"),
        ((x.transpose(2, 3), None), dict(out=_bf(1, 8, 64, 2)), ValueError, "dense in its last"),
    ]:
        with pytest.raises(error, match=message):
            kda.gated_norm(*args, **kw)


def test_rope_frequencies():
    f, a = kda.rope_frequencies(8, 100.0, device="cpu")
    assert a == 1.0 and f.dtype == torch.float64
    assert f.tolist() == pytest.approx([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], rel=1e-14)
    assert kda.rope_frequencies(8, 100.0, scaling="linear", factor=4.0, device="cpu")[0].tolist() == \
        pytest.approx((f / 4).tolist(), rel=1e-14)
    b, a = kda.rope_frequencies(8, 100.0, scaling="base", factor=4.0, device="cpu")
    assert a == 1.0 and float(b[0]) == 1.0 and float(b[3]) == pytest.approx(float(f[3]) / 4, rel=1e-12)
    assert bool((b[1:3] < f[1:3]).all()) and bool((b[1:3] > f[1:3] / 4).all())
    f, _ = kda.rope_frequencies(128, device="cpu")
    y, a = kda.rope_frequencies(128, scaling="ramp", factor=8.0, original_positions=4096, device="cpu")
    assert a == pytest.approx(0.1 * math.log(8) + 1, rel=1e-14)
    turns = 4096 * f / (2 * math.pi)
    ratio = y / f
    assert bool((ratio[turns > 40] == 1).all())
    assert ratio[turns < 0.8].tolist() == pytest.approx([1 / 8] * int((turns < 0.8).sum()))
    assert bool((ratio[1:] <= ratio[:-1]).all())
    for kw, message in [(dict(scaling="other"), "not one of"), (dict(factor=0.5), "at least 1"),
                        (dict(scaling="ramp", factor=2.0), "original_positions"), (dict(base=1.0), "base")]:
        with pytest.raises(ValueError, match=message):
            kda.rope_frequencies(128, device="cpu", **kw)
    for r in (0, 7):
        with pytest.raises(ValueError, match="even"):
            kda.rope_frequencies(r, device="cpu")
    with pytest.raises(ValueError, match="at least 4"):
        kda.rope_frequencies(2, scaling="base", factor=2.0, device="cpu")


def test_references_agree_with_closed_forms():
    """The 64-bit forms the GPU tests compare with, on cases worked out by hand."""
    from tests import ops_reference as ref
    one = torch.ones(3, 1, 2)
    o, S, mag, smag = ref.lin_attn(one, one, one, torch.log(torch.tensor([0.5])), [3],
                                   torch.full((1, 1, 2, 2), 8.0), [1], 1.0)
    assert o[:, 0, 0].tolist() == pytest.approx([10.0, 7.0, 5.5]) and float(S[0, 0, 0, 0]) == pytest.approx(2.75)
    assert mag.equal(o) and smag.equal(S)
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    f = torch.tensor([math.pi / 2, math.pi], dtype=torch.float64)
    p = torch.tensor([1])
    assert ref.rope(x, p, f, "half", 1.0)[0, 0].tolist() == pytest.approx([-3, -2, 1, -4, 9])
    assert ref.rope(x, p, f, "interleaved", 2.0)[0, 0].tolist() == pytest.approx([-4, 2, -6, -8, 9])
    back = ref.rope(ref.rope(x, p, f, "half", 1.0), p, f, "half", 1.0, inverse=True)
    assert back[0, 0].tolist() == pytest.approx(x[0, 0].tolist())
    y = ref.gated_norm(torch.tensor([[[3.0, 4.0]]]), torch.tensor([1.0, 2.0]), torch.zeros(1, 1, 2), "sigmoid", 0.0)
    assert y[0, 0].tolist() == pytest.approx([3 / math.sqrt(12.5) / 2, 4 / math.sqrt(12.5)])
