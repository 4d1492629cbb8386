"""CPU tests of which overlaps of their tensors the operators refuse.  The addresses are
made up and never touched: every case is refused by one check or another before any CUDA
call, and the message tells which."""
import pytest

from tests.test_ops_host import BASE, lib, norm_abi, rope_abi  # noqa: F401  (lib is a fixture)

ROW = 128 * 2  # bytes of a row
M = 1 << 24


def rope(lib, a, b):  # noqa: F811
    """kda_rope's answer for two tensors (in, out, strides, heads); where it finds no
    overlap, it goes on to the missing positions."""
    return rope_abi(lib, [a, b], pos=None)


def view(base, heads=4, st=512, sh=128):
    return base, st, sh, heads


def pair(x, y):
    (i, ist, ish, h), (o, ost, osh, _) = x, y
    return i, o, ist, ish, ost, osh, h


Q, K, QO, KO = (view(BASE + i * M) for i in range(4))


@pytest.mark.parametrize("q,k,message", [
    (pair(Q, K), pair(K, KO), "out of tensor 0 overlaps the in of tensor 1"),
    (pair(Q, QO), pair(K, Q), "out of tensor 1 overlaps the in of tensor 0"),
    (pair(Q, QO), pair(K, QO), "the outs of the two tensors overlap"),
    (pair(Q, Q), pair(Q, Q), "out of tensor 0 overlaps the in of tensor 1"),
    (pair(Q, view(BASE + M + 95 * 4 * ROW)), pair(K, KO), "out of tensor 0 overlaps the in of tensor 1"),
    # one head of a fused projection more than lies before the other's
    (pair(view(BASE, 4, 768), view(BASE, 4, 768)), pair(view(BASE + 3 * ROW, 2, 768), view(BASE + 3 * ROW, 2, 768)),
     "out of tensor 0 overlaps the in of tensor 1"),
    # token strides without a common step between the rows
    (pair(view(BASE, 1, 384), view(BASE, 1, 384)), pair(view(BASE + ROW, 1, 256), view(BASE + ROW, 1, 256)),
     "out of tensor 0 overlaps the in of tensor 1"),
])
def test_rope_refuses_tensors_in_each_other(lib, q, k, message):  # noqa: F811
    rc, err = rope(lib, q, k)
    assert rc == -1 and message in err, (rc, err)


@pytest.mark.parametrize("q,k", [
    (pair(Q, QO), pair(K, KO)),
    (pair(Q, Q), pair(K, K)),
    # views of one projection's output: side by side, and heads by turns
    (pair(view(BASE, 4, 768), view(BASE, 4, 768)), pair(view(BASE + 4 * ROW, 2, 768), view(BASE + 4 * ROW, 2, 768))),
    (pair(view(BASE, 4, 1024, 256), view(BASE, 4, 1024, 256)),
     pair(view(BASE + ROW, 4, 1024, 256), view(BASE + ROW, 4, 1024, 256))),
    # [heads][tokens][128], one tensor's heads behind the other's
    (pair(view(BASE, 4, 128, 96 * 128), view(BASE, 4, 128, 96 * 128)),
     pair(view(BASE + 4 * 96 * ROW, 2, 128, 96 * 128), view(BASE + 4 * 96 * ROW, 2, 128, 96 * 128))),
    # and by turns with them
    (pair(view(BASE, 4, 128, 2 * 96 * 128), view(BASE, 4, 128, 2 * 96 * 128)),
     pair(view(BASE + 96 * ROW, 4, 128, 2 * 96 * 128), view(BASE + 96 * ROW, 4, 128, 2 * 96 * 128))),
    # a tensor without heads overlaps nothing
    (pair(Q, Q), pair(view(BASE, 0), view(BASE, 0))),
])
def test_rope_takes_tensors_beside_each_other(lib, q, k):  # noqa: F811
    rc, err = rope(lib, q, k)
    assert rc == -1 and "are required" in err, (rc, err)


# Views of one buffer and one-entry dimensions in a single tensor.  gated_norm goes on to
# the weight, which overlaps the out here, where it finds no other overlap.
def norm(lib, **over):  # noqa: F811
    return norm_abi(lib, **dict(dict(w=over.get("out", BASE)), **over))


@pytest.mark.parametrize("over", [
    # in place on one half of a fused [x | gate], and of [gate | x]
    dict(x=BASE, gate=BASE + 4 * ROW, out=BASE, x_st=1024, g_st=1024, o_st=1024),
    dict(x=BASE + 4 * ROW, gate=BASE, out=BASE + 4 * ROW, x_st=1024, g_st=1024, o_st=1024),
    # x and gate by turns in each head
    dict(x=BASE, gate=BASE + ROW, out=BASE, x_st=1024, g_st=1024, o_st=1024, x_sh=256, g_sh=256, o_sh=256),
    # out in a third part of the buffer
    dict(x=BASE, gate=BASE + 4 * ROW, out=BASE + 8 * ROW, x_st=1536, g_st=1536, o_st=1536),
    # the stride of a dimension of one entry says nothing
    dict(x=BASE, out=BASE, T=1, x_st=512, o_st=4096),
    dict(x=BASE, out=BASE, H=1, x_sh=128, o_sh=640),
])
def test_gated_norm_takes_views_beside_each_other(lib, over):  # noqa: F811
    rc, err = norm(lib, **over)
    assert rc == -1 and "out overlaps weight" in err, (rc, err)


@pytest.mark.parametrize("over,message", [
    (dict(x=BASE, gate=BASE + 3 * ROW, out=BASE, x_st=1024, g_st=1024, o_st=1024), "out overlaps gate"),
    (dict(x=BASE, gate=BASE + 4 * ROW, out=BASE, x_st=1024, g_st=768, o_st=1024), "out overlaps gate"),
    (dict(x=BASE, gate=BASE, out=BASE), "out overlaps gate"),
    (dict(x=BASE, gate=BASE + M, out=BASE + 2 * ROW, x_st=1024, o_st=1024), "out overlaps x"),
    (dict(x=BASE, gate=BASE + M, out=BASE, x_st=1024, o_st=512), "out overlaps x"),
])
def test_gated_norm_refuses_rows_in_each_other(lib, over, message):  # noqa: F811
    rc, err = norm(lib, **over)
    assert rc == -1 and message in err, (rc, err)


@pytest.mark.parametrize("x,y", [
    # from one part of a fused buffer to another, and over a dimension of one entry
    (view(BASE, 2, 768), view(BASE + 2 * ROW, 2, 768)),
    (view(BASE, 1, 512, 128), view(BASE, 1, 512, 640)),
])
def test_rope_takes_views_beside_each_other(lib, x, y):  # noqa: F811
    rc, err = rope_abi(lib, [pair(x, y)], pos=None)
    assert rc == -1 and "are required" in err, (rc, err)
