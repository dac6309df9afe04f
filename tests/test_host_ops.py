"""Host side of the dense layer and AdamW: configurations refused without a GPU, constants of
the binding as the header has them."""
import os
import re

import pytest

import qml_gradients_amd as hq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _lib():
    if not os.path.exists(hq.LIB_PATH):
        from qml_gradients_amd import build
        build.build()
    return hq.load()


@pytest.mark.parametrize("bad", [dict(in_features=0), dict(in_features=(1 << 20) + 1), dict(out_features=-1),
                                 dict(max_batch=0), dict(max_batch=(1 << 24) + 1), dict(dtype=2), dict(dtype=7),
                                 dict(activation=6), dict(activation=-1), dict(alpha=float("inf")),
                                 dict(alpha=float("nan")), dict(device=-1)])
def test_dense_configurations_refused(bad):
    _lib()
    good = dict(in_features=8, out_features=4, max_batch=2)
    assert hq.hqml_dense_workspace_bytes(hq.make_dense_config(**good)) > 0
    cfg = hq.make_dense_config(**{**good, **bad})
    assert hq.hqml_dense_workspace_bytes(cfg) == 0
    with pytest.raises(hq.HqmlError) as e:
        hq.hqml_dense_create(cfg)
    assert e.value.status == hq.HQML_ERR_ARG


def test_null_arguments_refused():
    lib = _lib()
    assert lib.hqml_dense_workspace_bytes(None) == 0
    assert lib.hqml_dense_create(None, None) == hq.HQML_ERR_ARG
    assert lib.hqml_dense_destroy(None) == hq.HQML_OK
    assert lib.hqml_dense_forward(None, 1, None, 1, None, 1, None, None, 0, None, 1, None) == hq.HQML_ERR_ARG
    assert lib.hqml_dense_backward(None, 1, None, 1, None, 1, None, 1, None, None, 1, None, None) == hq.HQML_ERR_ARG
    assert lib.hqml_adamw_step(None, 0, None) == hq.HQML_ERR_ARG


def test_binding_constants_match_header():
    header = open(os.path.join(ROOT, "include", "hqml.h")).read()
    for name in re.findall(r"\b(HQML_(?:DTYPE|ACT|MOMENTS)_[A-Z0-9]+) = (\d+)", header):
        assert getattr(hq, name[0]) == int(name[1])
    assert "#define HQML_ADAMW_BLOCK %d" % hq.HQML_ADAMW_BLOCK in header
    assert hq.HQML_DENSE_MAX_FEATURES == 1 << 20 and "#define HQML_DENSE_MAX_FEATURES (1 << 20)" in header
    assert hq.HQML_DENSE_MAX_BATCH == 1 << 24 and "#define HQML_DENSE_MAX_BATCH (1 << 24)" in header
