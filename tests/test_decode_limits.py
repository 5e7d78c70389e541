"""Sizes whose products pass 32 bits in the decoder-layer calls (include/bq_decode.h), refused before any launch (the
fake pointers are never dereferenced)."""

import os

import pytest

import quantized_mixed_precision_gb300 as bq

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bq.LIB_PATH):
        from quantized_mixed_precision_gb300 import build
        build.build()
    return bq.lib()


@pytest.mark.parametrize("T,hq", [(1 << 24, 128), (1 << 24, 65536), (1 << 15, 65536)])
def test_too_many_query_rows(lib, T, hq):
    """Query rows (tokens times heads) are counted in 32 bits."""
    args = [FAKE, hq * 64, T, hq, 1, 64, FAKE, FAKE, 1 << 12, 64, 64, FAKE, 1 << 11, FAKE, FAKE, 1, T, 1 << 17, 0.1, 0,
            FAKE, None, FAKE, 1 << 62, None]
    assert lib.bq_attn_kv4(*args) == bq.BQ_ERR_UNSUPPORTED
