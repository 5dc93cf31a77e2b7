"""The attention step's entry points without a GPU: the library refuses what
the host can see before it touches the device, and the binding refuses wrong
memory, types, shapes and sizes before it calls the library."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from tenant_composite_lora_gb300 import build, native
    build.build()
    return native.load()


def test_library_refuses_null_and_bad_sizes(lib):
    out = ctypes.c_void_p()
    fake = 1 << 20  # aligned, never read: every call below returns before the device
    new = lambda *a: lib.lora_kv_cache_create(*a, ctypes.byref(out))
    assert lib.lora_kv_cache_create(4, 16, 2, 64, fake, fake, None) == 1
    assert new(4, 16, 2, 64, None, fake) == 1 and new(4, 16, 2, 64, fake, None) == 1
    assert new(0, 16, 2, 64, fake, fake) == 1 and new(4, 16, 0, 64, fake, fake) == 1
    assert new(4, 16, 2, 64, fake + 8, fake) == 1  # not 16-byte aligned
    for bad in ((4, 24, 2, 64), (4, 8, 2, 64), (4, 16, 2, 96), (4, 16, 257, 64), (1 << 24, 128, 1, 64)):
        assert new(*bad, fake, fake) == 5, bad
    assert out.value is None
    assert lib.lora_kv_cache_destroy(None) == 0 and lib.lora_attn_plan_destroy(None) == 0
    assert new(4, 16, 2, 64, fake, fake) == 0
    c = out.value

    def append(T=3, k=fake, ks=128, v=fake, vs=128, q=fake, qs=256, o=fake, os=256, hq=4, slots=fake, pos=fake,
               rope=fake, max_pos=8, rot=64, style=0):
        return lib.lora_kv_append(c, k, ks, v, vs, q, qs, o, os, hq, slots, pos, rope, max_pos, rot, style, T, None,
                                  None)

    for bad in (dict(T=-1), dict(k=None), dict(v=None), dict(slots=None), dict(pos=None), dict(rope=None),
                dict(max_pos=0), dict(rot=72), dict(rot=80), dict(rot=-16), dict(style=2), dict(ks=120), dict(vs=132),
                dict(k=fake + 2), dict(o=None), dict(hq=0), dict(qs=248), dict(os=260), dict(qs=264), dict(q=fake + 8)):
        assert append(**bad) == 1, bad
    assert append(hq=1025, qs=1 << 20, os=1 << 20) == 5 and append(T=(1 << 24) + 1) == 5
    assert append(T=0) == 0
    assert lib.lora_kv_append(None, fake, 128, fake, 128, None, 0, None, 0, 0, fake, None, None, 0, 0, 0, 1, None,
                              None) == 1
    assert lib.lora_kv_cache_destroy(c) == 0

    plan = lambda *a: lib.lora_attn_plan_create(*a, ctypes.byref(out))
    for bad in ((0, 1, 1, 1, 1, 4, 2, 64, 16), (1, -1, 1, 1, 1, 4, 2, 64, 16), (1, 1, 0, 1, 1, 4, 2, 64, 16),
                (1, 1, 1, -1, 1, 4, 2, 64, 16), (1, 1, 1, 1, 1, 5, 2, 64, 16), (1, 1, 1, 1, 1, 0, 2, 64, 16)):
        assert plan(*bad) == 1, bad
    for bad in ((1, 1, 1, 1, 1, 4, 2, 80, 16), (1, 1, 1, 1, 1, 4, 2, 64, 20), (1, 1, 1, 1, 1, 2048, 2, 64, 16),
                (1 << 25, 1, 1, 1, 1, 4, 2, 64, 16)):
        assert plan(*bad) == 5, bad
    assert lib.lora_attn_plan_create(1, 1, 1, 1, 1, 4, 2, 64, 16, None) == 1
    assert lib.lora_attn_plan_build(None, fake, fake, fake, 1, None, None, None, 0, 1, 0, 1, 4, None) == 1
    assert lib.lora_prefix_attention(fake, 256, fake, 256, None, None, None, 1.0, None) == 1
    assert lib.lora_attn_plan_status(None, None, ctypes.byref(ctypes.c_int())) == 1

    def sample(logits=fake, kind=0, stride=32, T=2, V=32, u=fake, tok=fake):
        return lib.lora_sample(logits, kind, stride, T, V, u, None, None, None, None, tok, None, None)

    for bad in (dict(logits=None), dict(u=None), dict(tok=None), dict(kind=2), dict(stride=31), dict(V=0), dict(T=-1),
                dict(logits=fake + 2), dict(kind=1, logits=fake + 1)):
        assert sample(**bad) == 1, bad
    assert sample(V=(1 << 20) + 1, stride=1 << 21) == 5 and sample(T=(1 << 24) + 1) == 5
    assert sample(T=0) == 0


def test_wrappers_refuse_before_the_library():
    import tenant_composite_lora_gb300 as tcl
    bf = torch.bfloat16
    with pytest.raises(ValueError, match="k must be"):
        tcl.LoraKvCache(2, 16, 2, 64, k=torch.zeros(2, 16, 2, 64, dtype=bf), device="cpu")
    with pytest.raises(ValueError, match="a CUDA tensor"):
        tcl.LoraKvCache(2, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="k holds"):
        tcl.lora_kv_cache_create(2, 16, 2, 64, torch.zeros(8, dtype=bf), None)

    class Cache:
        n_kv_heads, head_dim, handle = 2, 64, 1

    class Plan:
        TQ, n_q_heads, head_dim, handle = 3, 4, 64, 1

    x = torch.zeros(3, 2, 64, dtype=bf)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="k: a CUDA tensor"):
        tcl.kv_append(Cache, x, x, i32(3))
    with pytest.raises(ValueError, match="q: a CUDA tensor"):
        tcl.prefix_attention(torch.zeros(3, 4, 64, dtype=bf), Cache, Plan)
    with pytest.raises(ValueError, match="slots holds 2 entries, at least 3"):
        tcl.lora_kv_append(1, 0, 0, 0, 0, 0, 0, 0, 0, 0, i32(2), None, None, 0, 0, 0, 3)
    with pytest.raises(ValueError, match="rope holds 64 entries, at least 512"):
        tcl.lora_kv_append(1, 0, 0, 0, 0, 0, 0, 0, 0, 0, i32(3), i32(3), torch.zeros(64), 8, 64, 0, 3)

    class Unbuilt(tcl.LoraAttnPlan):
        def __init__(self):
            self.handle, self.TQ = 1, 0

        def close(self):
            self.handle = None

    p = Unbuilt()
    with pytest.raises(ValueError, match="3 requests, but 2 suffix lengths"):
        p.build(i32(4), i32(2), i32(3, 5), 3, 9)
    with pytest.raises(ValueError, match="suffix_pages is 2-D"):
        p.build(i32(4), i32(3), i32(15), 3, 9)
    with pytest.raises(ValueError, match="go together"):
        p.build(i32(4), i32(3), i32(3, 5), 3, 9, group_offsets=i32(2))
    with pytest.raises(ValueError, match="1 groups, but 2 prefix lengths"):
        p.build(i32(4), i32(3), i32(3, 5), 3, 9, i32(2), i32(2), i32(1, 4))
    with pytest.raises(ValueError, match="q_offsets: a CUDA tensor"):
        p.build(i32(4), i32(3), i32(3, 5), 3, 9)
    with pytest.raises(ValueError, match="lora_attn_plan_build: prefix_pages holds 3"):
        tcl.lora_attn_plan_build(1, i32(4), i32(3), i32(15), 5, i32(2), i32(1), i32(3), 4, 3, 1, 3, 9)
    with pytest.raises(ValueError, match="logits are 2-D"):
        tcl.sample(torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="lora_sample: top_p holds 1"):
        tcl.lora_sample(1 << 20, 0, 8, 2, 8, torch.zeros(2), None, None, torch.zeros(1), None, i32(2))
