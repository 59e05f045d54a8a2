"""Names of the package that callers may hold: the C ABI's type and status codes."""
import lm_head_logits_amd as L
from lm_head_logits_amd import _lib


def test_codes_are_attributes_of_the_package():
    for name in ("LMHEAD_BF16", "LMHEAD_F16", "LMHEAD_F32", "OK", "NOT_HANDLED", "PATH_AUTO", "PATH_NONE",
                 "PATH_SKINNY", "PATH_TILED", "PATH_NVFP4"):
        assert getattr(L, name) == getattr(_lib, name), name


def test_public_names():
    for name in L.__all__:
        assert hasattr(L, name), name
    assert issubclass(L.NotHandled, L.LmHeadError)
