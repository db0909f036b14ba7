"""Adapters, norms with rotation and prompt attention: refusals, which return before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from gguf_quant_integer_gb300 import build as xqbuild

FAKE = 1 << 20  # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def xq():
    xqbuild.build()
    from gguf_quant_integer_gb300 import xq as _xq
    _xq.lib()
    return _xq


def lora(xq, n_proj=1, n_inputs=1, M=1, ids=FAKE, x=FAKE, **kw):
    d = dict(type=30, n=4, rank=16, K=512, N=64, a=FAKE, b=FAKE, scales=FAKE, y=FAKE, input=0)
    d.update(kw)
    arr = (xq.xq_adapters * max(1, n_proj))(*[xq.xq_adapters(**d) for _ in range(max(1, n_proj))])
    ins = (ctypes.c_void_p * max(1, n_inputs))(*[x] * max(1, n_inputs))
    return xq.lib().xq_lora_add(arr, n_proj, ins, n_inputs, M, ids, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=8), 1), (dict(type=2), 1), (dict(input=1), 1), (dict(input=-1), 1), (dict(n_proj=17), 1), (dict(n_proj=-1), 1),
    (dict(n_inputs=65), 1), (dict(n_inputs=-1), 1), (dict(n_inputs=0), 1), (dict(x=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(y=None), 1),
    (dict(ids=None), 1), (dict(rank=0), 2), (dict(rank=12), 2), (dict(rank=264), 2), (dict(K=0), 2), (dict(K=40), 2), (dict(K=-32), 2),
    (dict(N=-1), 2), (dict(n=-1), 2), (dict(n=8193), 2), (dict(M=-1), 2), (dict(a=FAKE + 8), 3), (dict(b=FAKE + 2), 3), (dict(x=FAKE + 4), 3), (dict(y=FAKE + 2), 3),
    (dict(scales=FAKE + 1), 3), (dict(ids=FAKE + 2), 3), (dict(M=0, ids=None), 0), (dict(N=0, y=None), 0), (dict(n_proj=0), 0)])
def test_adapters(xq, kw, code):
    assert lora(xq, **kw) == code


def test_adapters_without_arrays(xq):
    L = xq.lib()
    assert L.xq_lora_add(None, 1, None, 0, 1, FAKE, None) == 1
    assert L.xq_lora_add(None, 0, None, 0, 1, None, None) == 0
    assert L.xq_lora_add((xq.xq_adapters * 1)(), 1, None, 1, 1, FAKE, None) == 1


def rope(xq, **kw):
    d = dict(type=0, y_type=30, tokens=3, heads=4, kv_heads=2, dim=128, q=FAKE, k=FAKE, q_stride=512, k_stride=256, q_out=2 * FAKE,
             k_out=2 * FAKE, q_out_stride=512, k_out_stride=256, q_weight=FAKE, k_weight=None, eps=1e-6, positions=FAKE, turns=FAKE, rot=128,
             pairs=0, magnitude=1.0)
    d.update(kw)
    return xq.lib().xq_qk_norm_rope(ctypes.byref(xq.xq_qk_rows(**d)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=8), 1), (dict(y_type=12), 1), (dict(pairs=2), 1), (dict(pairs=-1), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(q_out=None), 1),
    (dict(k_out=None), 1), (dict(positions=None), 1), (dict(turns=None), 1), (dict(tokens=-1), 2), (dict(heads=0), 2), (dict(kv_heads=0), 2),
    (dict(heads=1 << 17), 2), (dict(dim=80), 2), (dict(dim=0), 2), (dict(rot=-16), 2), (dict(rot=144), 2), (dict(rot=24), 2), (dict(eps=-1e-9), 2),
    (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2), (dict(magnitude=float("inf")), 2), (dict(q_stride=511), 2), (dict(k_stride=0), 2),
    (dict(q_out_stride=-512), 2), (dict(k_out_stride=255), 2), (dict(q=FAKE + 2), 3), (dict(k=FAKE + 1), 3), (dict(q_out=FAKE + 1), 3),
    (dict(k_out=FAKE + 1), 3), (dict(q_weight=FAKE + 2), 3), (dict(k_weight=FAKE + 3), 3), (dict(positions=FAKE + 4), 3), (dict(turns=FAKE + 4), 3),
    (dict(q_out=FAKE), 1), (dict(y_type=0, q_out=FAKE, q_out_stride=600), 1), (dict(tokens=0, q=None), 0)])
def test_norm_and_rotation(xq, kw, code):
    assert rope(xq, **kw) == code


def prompts(xq, **kw):
    d = dict(type=30, tokens=10, batch=1, heads=4, kv_heads=2, dim=128, q=FAKE, k=FAKE, v=FAKE, q_stride=512, k_stride=256, v_stride=256,
             out=2 * FAKE, starts=FAKE, scale=1.0, window=0)
    d.update(kw)
    return xq.xq_prompts(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(type=8), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(starts=None), 1), (dict(tokens=-1), 2),
    (dict(batch=-1), 2), (dict(heads=3), 2), (dict(heads=0), 2), (dict(kv_heads=0), 2), (dict(dim=32), 2), (dict(window=-1), 2),
    (dict(scale=float("nan")), 2), (dict(scale=-float("inf")), 2), (dict(q_stride=511), 2), (dict(k_stride=0), 2), (dict(v_stride=-256), 2),
    (dict(tokens=1 << 30, heads=2), 2), (dict(q=FAKE + 8), 3), (dict(k=FAKE + 2), 3), (dict(v=FAKE + 4), 3), (dict(out=FAKE + 8), 3),
    (dict(starts=FAKE + 2), 3), (dict(q_stride=516), 3), (dict(k_stride=257), 3), (dict(v_stride=260), 3), (dict(tokens=0, q=None), 0),
    (dict(batch=0, q=None), 0)])
@pytest.mark.parametrize("kind", [30, 1, 0])
def test_prompt_attention(xq, kw, code, kind):
    if kind == 0 and kw.get("q_stride") in (516,) or kind == 0 and kw.get("v_stride") == 260:
        code = None  # 16 bytes' multiples in fp32
    p = prompts(xq, **{"type": kind, **kw})
    if code is not None:
        assert xq.lib().xq_prompt_attn(ctypes.byref(p), FAKE, 1 << 40, None) == code


def test_prompt_attention_workspace(xq):
    L = xq.lib()
    size = lambda **kw: L.xq_prompt_attn_workspace_bytes(ctypes.byref(prompts(xq, **kw)))  # noqa: E731
    assert size() >= 16 and size(type=0) >= 16
    assert size(type=8) == 0 and size(heads=3) == 0 and size(dim=100) == 0 and L.xq_prompt_attn_workspace_bytes(None) == 0
    assert L.xq_prompt_attn(None, FAKE, 1 << 40, None) == 1
    assert L.xq_prompt_attn(ctypes.byref(prompts(xq)), FAKE + 4, 1 << 40, None) == 3


def test_packed_structures_have_the_structures_layout(xq):
    """The binding packs arguments as bytes: fields at the same places as the C structures'."""
    import struct
    for form, kind in (("@" + xq._ADAPTERS, xq.xq_adapters), ("@" + 3 * xq._ADAPTERS, xq.xq_adapters * 3)):
        assert struct.calcsize(form) == ctypes.sizeof(kind)
    values = list(range(1, 11))
    a = xq.xq_adapters.from_buffer_copy(struct.pack("@" + xq._ADAPTERS, *values))
    assert [getattr(a, f[0]) for f in a._fields_] == values
    values = [*range(1, 17), 0.5, 18, 19, 20, 1, 2.5]
    r = xq.xq_qk_rows.from_buffer_copy(xq._pack_rows(*values))
    assert [getattr(r, f[0]) for f in r._fields_] == values and len(xq._pack_rows(*values)) == ctypes.sizeof(r)
    values = [*range(1, 15), 0.25, 16]
    p = xq.xq_prompts.from_buffer_copy(xq._pack_prompts(*values))
    assert [getattr(p, f[0]) for f in p._fields_] == values and len(xq._pack_prompts(*values)) == ctypes.sizeof(p)


@pytest.mark.parametrize("clocks,code", [(0, 1), (-1, 1), ((1 << 32) + 1, 1), (1, 1), (1 << 32, 1)])
def test_stalled_prompt_attention(xq, clocks, code):
    assert xq.lib().xq_debug_stalled_prompt_attn(ctypes.byref(prompts(xq, q=None)), FAKE, 1 << 40, clocks, 1, None) == code
    assert xq.lib().xq_debug_stalled_prompt_attn(ctypes.byref(prompts(xq, tokens=0, q=None)), FAKE, 1 << 40, 1000, 1, None) == 0


@pytest.mark.parametrize("N,code", [((1 << 30) + 1, 2), ((1 << 31) - 1, 2), (1 << 30, 0)])
def test_adapters_of_very_many_columns(xq, N, code):
    """A step over the columns past 2^31 would be a negative column. (No rows: nothing is launched.)"""
    assert lora(xq, N=N, M=0 if code == 0 else 1) == code
