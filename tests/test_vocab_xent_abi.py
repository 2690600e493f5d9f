"""Cross entropy over a vocabulary: what the entry points refuse and how they plan, on the host, before anything is launched."""
import ctypes

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib as K
from attention_kl_divergence_streamkl_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.lib()


def ptr(off=0):
    return ctypes.c_void_p(0x10000000 + off)


SHAPE = dict(rows=4, vocab=100, channels=64, dtype=0, scale=1.0, hidden_stride=64, weight_stride=64)
FWD = dict(hidden=ptr(), weight=ptr(16), tokens=ptr(32), shape=None, loss=ptr(64), lse=ptr(128), ws=ptr(256), nbytes=1 << 20)
BWD = dict(hidden=ptr(), weight=ptr(16), tokens=ptr(32), lse=ptr(64), g=ptr(68), gl=None, shape=None, dh=ptr(128), dw=ptr(256),
           ws=ptr(512), nbytes=1 << 20)
BAD_SHAPES = [
    (dict(rows=-1), K.ERR_INVALID), (dict(vocab=0), K.ERR_INVALID), (dict(channels=0), K.ERR_INVALID),
    (dict(hidden_stride=56), K.ERR_INVALID), (dict(weight_stride=0), K.ERR_INVALID), (dict(scale=0.0), K.ERR_INVALID),
    (dict(scale=-1.0), K.ERR_INVALID), (dict(scale=float("nan")), K.ERR_INVALID), (dict(scale=float("inf")), K.ERR_INVALID),
    (dict(scale=3e38), K.ERR_INVALID),
    (dict(dtype=3), K.ERR_INVALID), (dict(dtype=-1), K.ERR_INVALID), (dict(dtype=2), K.ERR_UNSUPPORTED),
    (dict(channels=60), K.ERR_UNSUPPORTED), (dict(hidden_stride=68), K.ERR_UNSUPPORTED),
    (dict(weight_stride=68), K.ERR_UNSUPPORTED), (dict(rows=2**31), K.ERR_UNSUPPORTED), (dict(vocab=2**31), K.ERR_UNSUPPORTED),
    (dict(weight_stride=2**38), K.ERR_UNSUPPORTED),
]


def shape(**change):
    return K.XentShape(*{**SHAPE, **change}.values())


@pytest.mark.parametrize("change,code", BAD_SHAPES)
def test_shapes_that_are_refused(lib, change, code):
    s, n = shape(**change), ctypes.c_size_t(0)
    i = ctypes.c_int(0)
    assert lib.streamkl_vocab_xent_fwd(*{**FWD, "shape": s}.values(), None) == code
    assert lib.streamkl_vocab_xent_bwd(*{**BWD, "shape": s}.values(), None) == code
    assert lib.streamkl_vocab_xent_fwd_workspace(s, ctypes.byref(n)) == code
    assert lib.streamkl_vocab_xent_fwd_plan(s, 152, ctypes.byref(i), ctypes.byref(n)) == code
    assert lib.streamkl_vocab_xent_bwd_plan(s, 152, 1, 1, ctypes.byref(i), ctypes.byref(i), ctypes.byref(n)) == code


@pytest.mark.parametrize("change", [dict(hidden=None), dict(hidden=ptr(8)), dict(weight=None), dict(weight=ptr(4)),
                                    dict(tokens=None), dict(tokens=ptr(4)), dict(loss=None), dict(lse=ptr(2))])
def test_forward_refuses_pointers(lib, change):
    assert lib.streamkl_vocab_xent_fwd(*{**FWD, "shape": shape(), **change}.values(), None) == K.ERR_INVALID


@pytest.mark.parametrize("change", [dict(ws=None), dict(ws=ptr(8)), dict(nbytes=79)])
def test_forward_refuses_workspaces(lib, change):
    assert lib.streamkl_vocab_xent_fwd(*{**FWD, "shape": shape(), **change}.values(), None) == K.ERR_WORKSPACE


@pytest.mark.parametrize("rows,vocab,channels", [(1, 1, 8), (8, 131072, 4096), (333, 50021, 1000), (8192, 131072, 4096), (100, 20000, 4096),
                                                 (64, 32000, 4096), (5, 88, 496), (256, 19712, 512), (3000, 100, 64), (300, 12000, 520),
                                                 (100, 28000, 1024)])
def test_forward_plan(rows, vocab, channels):
    """Tiles of 160 to 256 columns in steps of 32, narrower ones only where that saves a part of a wave of 76 pairs."""
    B.build()
    width, nbytes = skl.vocab_xent_fwd_plan(rows, vocab, channels, 152)
    assert width in range(160, 257, 32)
    tiles, m = -(-vocab // width), -(-rows // 256)
    assert nbytes == -(-4 * rows // 256) * 256 + 2 * tiles * (-(-rows // 32) * 32) * 8

    def waves(w):
        return -(-m * -(-vocab // w) // 76)

    assert width == 256 or waves(width) * width < waves(256) * 256


@pytest.mark.parametrize("change", [dict(dh=None, dw=None), dict(dh=ptr(8)), dict(dw=ptr(8)), dict(hidden=None), dict(weight=None),
                                    dict(tokens=None), dict(lse=None), dict(g=None), dict(gl=ptr(2)),
                                    dict(dh=ptr()), dict(dw=ptr(16)), dict(dw=ptr()), dict(dh=ptr(16)), dict(dw=ptr(128))])
def test_backward_refuses_pointers(lib, change):
    assert lib.streamkl_vocab_xent_bwd(*{**BWD, "shape": shape(), **change}.values(), None) == K.ERR_INVALID


def test_no_rows_is_no_work(lib):
    s = shape(rows=0)
    assert lib.streamkl_vocab_xent_fwd(*{**FWD, "shape": s, "hidden": None, "ws": None}.values(), None) == K.OK
    assert lib.streamkl_vocab_xent_bwd(*{**BWD, "shape": s, "hidden": None, "dw": None, "ws": None}.values(), None) == K.OK


@pytest.mark.parametrize("rows,vocab,channels", [(1, 1, 8), (8, 131072, 4096), (333, 50021, 1000), (8192, 131072, 4096),
                                                 (1 << 20, 131072, 4096), (9000, 17001, 64), (4096, 1 << 20, 8192)])
def test_plan(rows, vocab, channels):
    """A piece of d is at most 512 MB or 8192 columns, the pieces cover the vocabulary, and the sums of dhidden are split
    only where its tiles are too few."""
    B.build()
    pieces, splits, nbytes = skl.vocab_xent_plan(rows, vocab, channels, 152)
    columns = -(-vocab // pieces)
    assert pieces >= 1 and (columns <= 8192 or 2 * rows * columns <= 1 << 29)
    tiles = -(-rows // 256) * -(-channels // 256)
    assert splits == 1 or splits * tiles <= 76
    _, _, without = skl.vocab_xent_plan(rows, vocab, channels, 152, want_dhidden=False)
    assert without <= nbytes
    if pieces > 1 or splits > 1:
        assert 0 <= nbytes - without - 4 * splits * rows * channels < 256
    _, _, alone = skl.vocab_xent_plan(rows, vocab, channels, 152, want_dweight=False)
    assert nbytes - alone == 2 * rows * channels  # room for a copy of hidden


@pytest.mark.parametrize("hidden,weight,tokens,error", [
    (torch.zeros(3, 8), torch.zeros(5, 8), torch.zeros(3, dtype=torch.int64), TypeError),
    (torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.float16), torch.zeros(3, dtype=torch.int64), TypeError),
    (torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(5, 16, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64), ValueError),
    (torch.zeros(3, 12, dtype=torch.bfloat16), torch.zeros(5, 12, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64), ValueError),
    (torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(0, 8, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64), ValueError),
    (torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64), ValueError),
    (torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16), torch.zeros(3), TypeError),
])
def test_binding_refuses(hidden, weight, tokens, error):
    B.build()
    with pytest.raises(error):
        skl.vocab_xent_fwd(hidden, weight, tokens)
