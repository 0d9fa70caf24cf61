"""Chunk attention's limits on heads and pages, refused on the host (nothing is launched)."""
import pytest

UNSUP = -2
fake = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def kvz():
    from decode_attention_value_gb300 import _build

    _build.build()
    import decode_attention_value_gb300 as m

    return m


@pytest.mark.parametrize("coded", [False, True])
def test_heads_and_pages_beyond_the_kernels_numbers(kvz, coded):
    lib = kvz.lib()

    def call(hkv, pages):
        head = (kvz.Dims(hkv, 128, 16), 1, hkv, fake, 1, fake, fake, 4, fake)
        own = (fake, fake, 9, fake, 1 << 20) if coded else ()
        fn = lib.kvz_chunk_attention if coded else lib.kvz_chunk_attention_raw
        return fn(*head, *own, fake, pages, 0, 0, fake, 1, fake, 1 << 40, fake, None)

    for hkv in (2 ** 20 + 1, 2 ** 23, 2 ** 24, 2 ** 27, 2 ** 31 - 1):  # a KV head's number shares a word with flags
        assert call(hkv, 1) == UNSUP
        assert lib.kvz_chunk_attention_workspace_size(kvz.Dims(hkv, 128, 16), 1, hkv, 1, 4, int(coded)) == 0
    for hkv, pages in ((8, 2 ** 23), (1, 2 ** 26), (8, 2 ** 55), (8, 2 ** 60), (8, 2 ** 63 - 1), (2 ** 20, 64)):
        assert call(hkv, pages) == UNSUP  # rows of the pool's tensor map, also where their number wraps in 64 bits
