"""The most work that a decode attention's tables may allow (no GPU: a call
within the limits goes on to the check of its buffers and fails there)."""
import pytest

import test_source_refusals as sources
from combine_attention_ffn_gb300 import afd


@pytest.fixture(scope="module")
def lib():
    from combine_attention_ffn_gb300 import build

    return afd.load_library(build.build())


@pytest.mark.parametrize("B,Hkv,G,tokens,refused", [
    (1 << 20, 1, 1, 1 << 30, True), (1 << 20, 8, 4, 1 << 22, True), (1 << 16, 16, 17, 1 << 25, True), (1 << 30, 1, 8, 1 << 16, True),
    (1 << 14, 1, 8, (1 << 30) - 16, False), (2048, 8, 16, 1 << 24, False), (1 << 20, 8, 8, 1 << 20, False), (1, 64, 8, (1 << 31) - 2048, False)])
def test_tokens_of_all_tables(lib, B, Hkv, G, tokens, refused):
    cache = sources._descriptor(num_kv_heads=Hkv, k_page_stride=Hkv * 16 * 128, v_page_stride=Hkv * 16 * 128)
    width = Hkv * G * 128
    status = sources._attend(lib, cache, B=B, Hq=Hkv * G, max_pages=tokens // 16, table_stride=tokens // 16, q_stride=width,
                             out_stride=width)
    assert status == (afd.ERR_UNSUPPORTED if refused else afd.ERR_ARG)
