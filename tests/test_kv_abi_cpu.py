"""Host-only checks of the paged key/value cache's entry points: sizes, and every refusal's status
and message.  No call reaches a GPU: each has one argument that validation refuses."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "hybrid_decode_replay_amd", "libreplayssm.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libreplayssm.so not built")

A = 0x10000          # an address that validation alone sees


def rb():
    from hybrid_decode_replay_amd import binding
    return binding


def refused(status, want):
    assert status == want, (status, rb().lib().replay_last_error())
    assert rb().lib().replay_last_error()


def cfg(**kw):
    c = rb().kv_config(8, 100, 16, 20)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def layer(**kw):
    b = rb()
    x = b.kv_layer(8, 2, 128, 100, 16, io_dtype=b.BF16, rot_dim=128)
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def test_pool_bytes():
    b = rb()
    assert b.kv_bytes(cfg()) == 4 * (64 + 7 * 64 + 8 * 20 + 100)
    assert b.kv_bytes(cfg(batch=65)) == 4 * (64 + 7 * 128 + 65 * 20 + 100)


@pytest.mark.parametrize("kw", [dict(batch=0), dict(batch=4097), dict(npages=0), dict(page_size=8), dict(page_size=48),
                                dict(page_size=512), dict(max_pages=0), dict(max_pages=1 << 26),
                                dict(batch=4096, max_pages=1 << 18), dict(abi_version=7)])
def test_pool_shapes(kw):
    b = rb()
    want = b.ERR_ARG if "abi_version" in kw else b.ERR_SHAPE
    c = cfg(**kw)
    assert b.kv_bytes(c) == 0
    refused(b.lib().replay_kv_reset(ctypes.byref(c), A, None), want)
    refused(b.lib().replay_kv_commit(ctypes.byref(c), A, None, None), want)
    refused(b.lib().replay_kv_release(ctypes.byref(c), A, None, None), want)
    refused(b.lib().replay_kv_reserve(ctypes.byref(c), A, 1, None, None, 8, A, A, None, None), want)
    with pytest.raises(b.ReplayError):
        b.KVPages(c)


def test_pool_pointers_and_counts():
    b, L = rb(), rb().lib()
    c = ctypes.byref(cfg())
    refused(L.replay_kv_reset(None, A, None), b.ERR_ARG)
    refused(L.replay_kv_reset(c, None, None), b.ERR_ARG)
    refused(L.replay_kv_reset(c, A + 16, None), b.ERR_ALIGN)
    refused(L.replay_kv_commit(c, A, A + 2, None), b.ERR_ALIGN)
    for args, want in [((1, None, None, 8, None, A, None), b.ERR_ARG), ((1, None, None, 8, A, None, None), b.ERR_ARG),
                       ((1, None, None, 8, A + 4, A, None), b.ERR_ALIGN), ((0, None, None, 8, A, A, None), b.ERR_CAPACITY),
                       ((17, None, None, 999, A, A, None), b.ERR_CAPACITY), ((2, None, None, 15, A, A, None), b.ERR_SHAPE),
                       ((1, None, None, 8, A, A, A), b.ERR_ARG), ((0, A, None, 8, A, A, None), b.ERR_ARG),
                       ((1, A, None, 8, A, A, A), b.ERR_ARG), ((0, A, None, 0, A, A, A), b.ERR_SHAPE),
                       ((0, A + 1, None, 8, A, A, A), b.ERR_ALIGN)]:
        refused(L.replay_kv_reserve(c, A, *args, None), want)


LAYERS = [(dict(io_dtype=1), "DTYPE"), (dict(cache_dtype=2), "DTYPE"), (dict(cache_dtype=5), "DTYPE"), (dict(nkv=0), "SHAPE"),
          (dict(nheads=7), "SHAPE"), (dict(nheads=1), "SHAPE"), (dict(nheads=8192), "SHAPE"), (dict(head_dim=96), "UNSUPPORTED"),
          (dict(page_size=24), "SHAPE"), (dict(npages=0), "SHAPE"), (dict(rot_dim=24), "SHAPE"), (dict(rot_dim=144), "SHAPE"),
          (dict(rot_dim=-16), "SHAPE"), (dict(rot_style=2), "ARG"), (dict(abi_version=0), "ARG")]


def append(**kw):
    a = rb().KVAppendArgs(q=A, k=A, v=A, q_stride=1536, k_stride=1536, v_stride=1536, slots=A, pos=A, freq=A, axis=None,
                          naxes=1, rows=4, q_out=A, K=A, V=A)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def attention(**kw):
    a = rb().KVAttentionArgs(q=A, q_stride=1024, K=A, V=A, table=A, end=A, batch=8, max_pages=20, ntok=1, window=0,
                             scale=1.0, o=A)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


@pytest.mark.parametrize("kw,code", LAYERS)
def test_layers(kw, code):
    b, L = rb(), rb().lib()
    want = getattr(b, "ERR_" + code)
    x = layer(**kw)
    refused(L.replay_kv_append(ctypes.byref(x), append(), None), want)
    refused(L.replay_kv_attention(ctypes.byref(x), attention(), A, 1 << 40, None), want)
    assert b.kv_attention_workspace(x, 8) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "SHAPE"), (dict(rows=(1 << 25) + 1), "SHAPE"), (dict(K=None), "ARG"), (dict(V=A + 8), "ALIGN"),
    (dict(k=None), "ARG"), (dict(v=A + 2), "ALIGN"), (dict(q=None), "ARG"), (dict(q_out=None), "ARG"), (dict(q_stride=1020), "ARG"),
    (dict(k_stride=255), "ARG"), (dict(v_stride=260), "ARG"), (dict(k_stride=1 << 31), "ARG"), (dict(slots=None), "ARG"),
    (dict(slots=A + 4), "ALIGN"), (dict(pos=None), "ARG"), (dict(freq=None), "ARG"), (dict(naxes=0), "SHAPE"),
    (dict(naxes=9), "SHAPE"), (dict(k_scale=A), "ARG"), (dict(v_scale=A), "ARG"), (dict(err=A + 2), "ALIGN")])
def test_append(kw, code):
    b = rb()
    refused(b.lib().replay_kv_append(ctypes.byref(layer()), append(**kw), None), getattr(b, "ERR_" + code))


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), "SHAPE"), (dict(batch=4097), "SHAPE"), (dict(max_pages=0), "SHAPE"), (dict(max_pages=1 << 27), "SHAPE"),
    (dict(ntok=0), "CAPACITY"), (dict(ntok=17), "CAPACITY"), (dict(window=-1), "ARG"), (dict(q=None), "ARG"), (dict(q=A + 8), "ALIGN"),
    (dict(q_stride=1016), "ARG"), (dict(q_stride=1028), "ARG"), (dict(K=None), "ARG"), (dict(V=None), "ARG"), (dict(o=None), "ARG"),
    (dict(o=A + 4), "ALIGN"), (dict(table=None), "ARG"), (dict(end=A + 2), "ALIGN"), (dict(lse=A + 2), "ALIGN"),
    (dict(k_scale=A, v_scale=A), "ARG"), (dict(batch=4096, max_pages=1 << 18), "SHAPE")])
def test_attention(kw, code):
    b = rb()
    refused(b.lib().replay_kv_attention(ctypes.byref(layer()), attention(**kw), A, 1 << 40, None), getattr(b, "ERR_" + code))


def test_attention_units_stay_in_32_bits():
    b = rb()
    wide = layer(nheads=4096, nkv=4096)
    refused(b.lib().replay_kv_attention(ctypes.byref(wide), attention(q_stride=4096 * 128, batch=4096, max_pages=1 << 17), A,
                                        1 << 60, None), b.ERR_SHAPE)


def test_scales_and_workspace():
    b, L = rb(), rb().lib()
    fp8 = layer(cache_dtype=b.FP8_E4M3)
    refused(L.replay_kv_append(ctypes.byref(fp8), append(), None), b.ERR_ARG)
    refused(L.replay_kv_attention(ctypes.byref(fp8), attention(k_scale=A), A, 1 << 40, None), b.ERR_ARG)
    n = b.kv_attention_workspace(layer(), 8, 1)
    assert n > 0 and n % 256 == 0
    refused(L.replay_kv_attention(ctypes.byref(layer()), attention(), None, n, None), b.ERR_ARG)
    refused(L.replay_kv_attention(ctypes.byref(layer()), attention(), A, n - 1, None), b.ERR_ALIGN)
    refused(L.replay_kv_attention(ctypes.byref(layer()), attention(), A + 64, n, None), b.ERR_ALIGN)
    refused(L.replay_kv_attention(ctypes.byref(layer()), None, A, n, None), b.ERR_ARG)
    refused(L.replay_kv_append(ctypes.byref(layer()), None, None), b.ERR_ARG)
    refused(L.replay_kv_append(None, append(), None), b.ERR_ARG)


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    b = rb()
    x = layer(rot_dim=0)
    K = torch.zeros(100, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        b.kv_attention(x, torch.zeros(1, 1024), K, K, torch.zeros(1, 1), torch.zeros(1))
    with pytest.raises(ValueError, match="device"):
        b.kv_append(x, K, K, torch.zeros(1, 256), torch.zeros(1, 256), torch.zeros(1))
    with pytest.raises(ValueError, match="device"):
        b.KVPages(cfg(), mem=torch.zeros(5000, dtype=torch.int32)).commit()
