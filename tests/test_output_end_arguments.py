"""Arguments of the output end's operators that are settled on the host (CPU only)."""

import pytest

from layer_optimizer_gb300 import build, native


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return native.load()


@pytest.mark.parametrize("piece", [1024, 1 << 20, 1 << 40, 2 ** 63 - 1024, 2 ** 63 - 512, 2 ** 63 - 256])
@pytest.mark.parametrize("n,d,v", [(100, 64, 1000), (17, 61, 1), (300, 256, 1023)])
def test_a_piece_beyond_the_vocabulary_is_the_whole_of_it(n, d, v, piece):
    # every size of at least V is one piece, up to the type's largest multiple of 256
    assert native.lce_vocab_workspace_bytes(n, d, v, piece) == native.lce_vocab_workspace_bytes(n, d, v, 1024)
