"""The calls that take their arguments as 64-bit words: a word that is no 32-bit number is refused
by its place, not cut to one that the call would accept."""
import struct

import pytest

import paged_kv_cache_154_gb300 as pa


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_154_gb300 import build
    build.build()


A = 0x10000
# what each call accepts with no tokens, and the places of its 32-bit words
CALLS = {
    "pa_rope": ("22q", [A, 1024, A, 1024, 8, A, 256, A, 256, 2, pa.PA_BF16, A, 64, 128, 0, A, 1, 0,
                        0, 0, 128, 0], [4, 9, 10, 12, 13, 14, 16, 18, 19, 20]),
    "pa_rope_append_kv": ("33q", [A, 1024, A, 1024, 8, 0, 0, A, 256, A, 256, pa.PA_BF16, A, A,
                                  pa.PA_BF16, A, A, A, A, A, A, 64, 128, 0, A, 1, 0, 0, 9, 2, 128,
                                  16, 0],
                          [4, 11, 14, 21, 22, 23, 25, 27, 28, 29, 30, 31]),
    "pa_prompt_attention": ("16qd3q", [A, 1024, A, 1024, A, 256, A, 256, pa.PA_BF16, A, 2, 0, 8, 8,
                                       2, 128, 0.1, 0, 0, 0], [8, 10, 11, 12, 13, 14, 15]),
}


@pytest.mark.parametrize("name", CALLS)
def test_words_outside_32_bits(name):
    form, words, small = CALLS[name]
    call = getattr(pa.lib(), name + "_packed")
    assert call(struct.pack(form, *words)) == 0
    for i in small:
        for beside in (1 << 32, -(1 << 32), 1 << 31, -(1 << 31) - 1 - words[i]):
            wrong = list(words)
            wrong[i] += beside
            if -(1 << 31) <= wrong[i] < 1 << 31:
                continue
            assert call(struct.pack(form, *wrong)) == 1
            assert f"argument {i}" in pa.lib().pa_last_error().decode()
    for i, w in enumerate(words):                  # strides and addresses are 64 bits
        if i not in small and not isinstance(w, float):
            more = list(words)
            more[i] += 1 << 40
            assert call(struct.pack(form, *more)) == 0
