"""kvz_append_tokens without a GPU: host-side refusals (nothing is launched) and the rotary
table, checked against its definition in long decimal arithmetic."""
import decimal

import pytest
import torch


@pytest.fixture(scope="module")
def kvz():
    from decode_attention_value_gb300 import _build

    _build.build()
    import decode_attention_value_gb300 as m

    return m


def test_host_rejects_bad_arguments(kvz):
    lib = kvz.lib()
    E = dict(inval=-1, unsup=-2, align=-3)
    fake = 1 << 20  # never dereferenced: every call below returns before any launch

    def app(hkv=8, d=128, p=16, T=4, hq=32, q=fake, qs=(4096, 128), k=fake, ks=(1024, 128), v=fake, vs=(1024, 128),
            slots=fake, pos=fake, axes=1, rope=fake, rot=128, flags=0, scale=1.0, q_out=fake, pool=fake, pages=9,
            status=fake):
        return lib.kvz_append_tokens(kvz.Dims(hkv, d, p), T, hq, q, *qs, k, *ks, v, *vs, slots, pos, axes, rope, rot,
                                     flags, scale, q_out, pool, pages, status, None)

    assert app(d=64) == E["unsup"]
    assert app(p=32) == E["unsup"]
    assert app(hkv=0) == E["inval"]
    assert app(T=0, q=None, k=None, v=None, slots=None, pool=None, rope=None, pos=None, status=None) == 0
    assert app(T=-1) == E["inval"]
    assert app(hq=-1) == E["inval"]
    assert app(pages=-1) == E["inval"]
    assert app(flags=2) == E["inval"]
    # rotated dimensions: multiples of 16 up to the head dimension
    assert app(rot=144) == E["inval"]
    assert app(rot=-16) == E["inval"]
    for rot in (8, 2, 120):
        assert app(rot=rot) == E["unsup"]
    assert app(axes=5) == E["unsup"]
    assert app(axes=0) == E["inval"]
    assert app(rope=None) == E["inval"]
    assert app(pos=None) == E["inval"]
    # k, v, slots and the pool go together; q, q_out and num_q_heads go together
    for name in ("k", "v", "slots", "pool", "q", "q_out", "status"):
        assert app(**{name: None}) == E["inval"], name
    assert app(hq=0) == E["inval"]
    assert app(q=None, q_out=None, hq=0, k=None, v=None, slots=None, pool=None) == E["inval"]
    # 16-byte vectors
    for name in ("q", "k", "v", "q_out", "pool", "rope"):
        assert app(**{name: fake + 8}) == E["align"], name
    for name in ("slots", "pos", "status"):
        assert app(**{name: fake + 2}) == E["align"], name
    for name in ("qs", "ks", "vs"):
        assert app(**{name: (1028, 128)}) == E["align"], name
        assert app(**{name: (1024, 132)}) == E["align"], name
        assert app(**{name: (-1024, 128)}) == E["align"], name
    assert app(T=(1 << 31) - 1) == E["unsup"]


def test_binding_rejects_bad_tensors(kvz):
    x = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):  # no tokens
        kvz.append_tokens(None, None, None, None, st)
    with pytest.raises(ValueError):  # values without keys
        kvz.append_tokens(None, x, None, None, st, q=x)


def test_rope_table_is_the_frequency_in_turns(kvz):
    decimal.getcontext().prec = 60
    pi = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    inv = torch.cat([500000.0 ** (-torch.arange(64, dtype=torch.float64) / 64),
                     torch.tensor([0.0, 3.0, 4.0, 6.5, 1e6, -0.25, 1e-9], dtype=torch.float64)])
    axis = torch.arange(inv.numel()) % 3
    table = kvz.rope_table(inv, axis)
    assert table.dtype == torch.int64 and table.shape == (inv.numel(), 2)
    assert torch.equal(table[:, 1], axis)
    assert torch.equal(kvz.rope_table(inv)[:, 1], torch.zeros_like(axis))
    for f, t in zip(inv.tolist(), table[:, 0].tolist()):
        turns = decimal.Decimal(f) / (2 * pi)
        want = int((turns * 2 ** 64).to_integral_value())
        off = (t - want + (1 << 63)) % (1 << 64) - (1 << 63)
        # the quotient is rounded to 53 bits of |turns| (pi and the division: 3 half steps), then to 2^-64
        assert abs(off) <= 3 * float(abs(turns)) * 2.0 ** (64 - 53) + 1024, (f, off)
    with pytest.raises(ValueError):
        kvz.rope_table(inv[None])
    with pytest.raises(ValueError):
        kvz.rope_table(inv, axis[:-1])


def test_caches_on_the_host_append(kvz):
    """A cache kept on the host takes tokens as they are and refuses to rotate them."""
    from decode_attention_value_gb300.cache import RawKVCache

    c = RawKVCache(2, 2, 3, 4, num_slots=9, device="cpu")
    c.admit(1, torch.zeros((2, 1, 2, 2, 16, 128), dtype=torch.bfloat16), 15)
    for step in range(3):  # past the page's end
        kv = torch.randn((2, 2, 2, 2, 128)).to(torch.bfloat16)
        q = torch.randn((2, 2, 4, 128)).to(torch.bfloat16)
        assert torch.equal(c.append([2, 1], kv, q=q), q)
        for i, slot in enumerate((2, 1)):
            n = int(c.lens[slot]) - 1
            assert torch.equal(c.pool[:, c.pages[slot][n // 16], :, :, n % 16], kv[:, i])
    assert c.lens[[1, 2]].tolist() == [18, 3]
    with pytest.raises(ValueError):
        c.append([0], kv[:, :1], rope=kvz.rope_table(torch.ones(64)))
