"""Host-only checks of the norm, E4M3 projection and prompt entry points: every refusal's status and message, the largest
sizes, the binding's own checks.  No call reaches a GPU: each has one argument that validation refuses."""
import ctypes
import os

import pytest

from test_kv_abi_cpu import A, LIB, rb, refused

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libreplayssm.so not built")


def with_(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def norm(**kw):
    b = rb()
    return with_(b.NormArgs(b.ABI_VERSION, b.BF16, b.FP8_E4M3, 4, 1, 256, 1e-6, x=A, x_stride=256, res=A, res_stride=256,
                            weight=A, sum=A + 4096, y=A, y_scale=A), kw)


NORMS = [(dict(abi_version=2), "ARG"), (dict(io_dtype=1), "DTYPE"), (dict(io_dtype=4), "DTYPE"), (dict(y_dtype=2), "DTYPE"),
         (dict(y_dtype=1), "DTYPE"), (dict(n=0), "SHAPE"), (dict(n=136), "SHAPE"), (dict(n=16512), "SHAPE"),
         (dict(y_dtype=3, y_scale=None, n=12), "SHAPE"), (dict(heads=0), "SHAPE"), (dict(heads=1 << 23), "SHAPE"),
         (dict(rows=-1), "SHAPE"), (dict(rows=1 << 26), "SHAPE"), (dict(rows=1 << 24, n=2048, x_stride=2048, res_stride=2048), "SHAPE"),
         (dict(rows=1 << 20, heads=64), "SHAPE"), (dict(eps=-1.0), "ARG"), (dict(eps=float("nan")), "ARG"), (dict(x=None), "ARG"),
         (dict(x=A + 8), "ALIGN"), (dict(x_stride=248), "ARG"), (dict(x_stride=260), "ARG"), (dict(x_stride=1 << 31), "ARG"),
         (dict(res=A + 2), "ALIGN"), (dict(res_stride=255), "ARG"), (dict(sum=A + 8), "ALIGN"), (dict(res=None), "ARG"),
         (dict(sum=A, res_stride=264), "ARG"), (dict(weight=A + 4), "ALIGN"), (dict(y=None), "ARG"), (dict(y=A + 8), "ALIGN"),
         (dict(y_scale=None), "ARG"), (dict(y_scale=A + 2), "ALIGN"), (dict(y_dtype=3), "ARG")]


@pytest.mark.parametrize("kw,want", NORMS)
def test_norm_refusals(kw, want):
    b = rb()
    refused(b.lib().replay_norm(norm(**kw), None), getattr(b, "ERR_" + want))


def linear(**kw):
    b = rb()
    return with_(b.LinearFP8Args(b.ABI_VERSION, b.BF16, 4, 256, 100, x=A, x_stride=256, x_scale=A, w=A, w_scale=A, y=A,
                                 y_stride=100), kw)


LINEARS = [(dict(abi_version=0), "ARG"), (dict(y_dtype=1), "DTYPE"), (dict(y_dtype=4), "DTYPE"), (dict(k=0), "SHAPE"),
           (dict(k=64), "SHAPE"), (dict(k=200), "SHAPE"), (dict(k=(1 << 20) + 128), "SHAPE"), (dict(n=0), "SHAPE"),
           (dict(n=(1 << 24) + 1), "SHAPE"), (dict(m=-1), "SHAPE"), (dict(m=(1 << 24) + 1), "SHAPE"),
           (dict(m=1 << 20, n=1 << 20, y_stride=1 << 20), "SHAPE"), (dict(x=None), "ARG"), (dict(x=A + 8), "ALIGN"),
           (dict(x_stride=128), "ARG"), (dict(x_stride=264), "ARG"), (dict(x_scale=None), "ARG"), (dict(x_scale=A + 2), "ALIGN"),
           (dict(w=None), "ARG"), (dict(w=A + 4), "ALIGN"), (dict(w_scale=None), "ARG"), (dict(w_scale=A + 1), "ALIGN"),
           (dict(y=None), "ARG"), (dict(y=A + 1), "ALIGN"), (dict(y_stride=99), "ARG"), (dict(y_stride=1 << 31), "ARG")]


@pytest.mark.parametrize("kw,want", LINEARS)
def test_linear_refusals(kw, want):
    b = rb()
    refused(b.lib().replay_linear_fp8(linear(**kw), None), getattr(b, "ERR_" + want))


def prefill(**kw):
    b = rb()
    return with_(b.GDNPrefillArgs(b.ABI_VERSION, b.BF16, 4, 2, 128, 128, 3, 100, 1.0, starts=A, q=A, k=A, v=A, q_stride=256,
                                  k_stride=256, v_stride=512, alpha=A, beta=A, S_in=A, S_out=A, o=A), kw)


SIZES = [(dict(abi_version=3), "ARG"), (dict(io_dtype=2), "DTYPE"), (dict(io_dtype=4), "DTYPE"), (dict(nheads=0), "SHAPE"),
         (dict(nheads=5), "SHAPE"), (dict(nheads=8192), "SHAPE"), (dict(ngroups=0), "SHAPE"), (dict(head_dim=0), "SHAPE"),
         (dict(head_dim=24), "SHAPE"), (dict(head_dim=272), "SHAPE"), (dict(state_dim=96), "SHAPE"), (dict(state_dim=512), "SHAPE"),
         (dict(nseq=0), "SHAPE"), (dict(nseq=4097), "SHAPE"), (dict(nseq=4096, nheads=256), "SHAPE"), (dict(rows=-1), "SHAPE"),
         (dict(rows=(1 << 30) + 1), "SHAPE")]
POINTERS = [(dict(starts=None), "ARG"), (dict(starts=A + 2), "ALIGN"), (dict(q=None), "ARG"), (dict(k=A + 8), "ALIGN"),
            (dict(v=None), "ARG"), (dict(q_stride=248), "ARG"), (dict(k_stride=260), "ARG"), (dict(v_stride=256), "ARG"),
            (dict(v_stride=1 << 31), "ARG"), (dict(alpha=None), "ARG"), (dict(beta=A + 2), "ALIGN"), (dict(S_in=A + 8), "ALIGN"),
            (dict(S_out=A + 4), "ALIGN"), (dict(o=None), "ARG"), (dict(o=A + 8), "ALIGN")]


@pytest.mark.parametrize("kw,want", SIZES + POINTERS)
def test_prefill_refusals(kw, want):
    b = rb()
    L = b.lib()
    refused(L.replay_gdn_prefill(prefill(**kw), A * 16, 1 << 40, None), getattr(b, "ERR_" + want))
    if (kw, want) in SIZES:
        assert L.replay_gdn_prefill_workspace(prefill(**kw)) == 0 and L.replay_last_error()


def test_null_arguments():
    b = rb()
    L = b.lib()
    refused(L.replay_norm(None, None), b.ERR_ARG)
    refused(L.replay_linear_fp8(None, None), b.ERR_ARG)
    refused(L.replay_gdn_prefill(None, None, 0, None), b.ERR_ARG)
    assert L.replay_gdn_prefill_workspace(None) == 0


def test_calls_without_rows_launch_nothing():
    b = rb()
    assert b.lib().replay_norm(norm(rows=0, x=None, y=None), None) == b.OK
    assert b.lib().replay_linear_fp8(linear(m=0, x=None, y=None), None) == b.OK


def test_the_binding_refuses_host_tensors_and_mixed_arguments():
    torch = pytest.importorskip("torch")
    b = rb()
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        b.norm(x)
    codes = torch.zeros((2, 256), dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="device tensors"):
        b.linear_fp8(codes, torch.zeros(2, 2), codes, torch.zeros(1, 2))
    g = torch.zeros(2, 2)
    with pytest.raises(ValueError, match="device tensors"):
        b.gdn_prefill(x, x, x, g, g, torch.zeros(2, dtype=torch.int32))


def test_structures_match_the_header():
    """Sizes of the argument blocks as a C compiler lays them out."""
    import subprocess
    import tempfile
    b = rb()
    src = ('#include "replayssm.h"\n#include <stdio.h>\nint main(void){printf("%zu %zu %zu\\n", sizeof(replay_norm_args), '
           'sizeof(replay_linear_fp8_args), sizeof(replay_gdn_prefill_args));return 0;}\n')
    with tempfile.TemporaryDirectory() as d:
        with open(os.path.join(d, "s.c"), "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I", os.path.dirname(b.HEADER), "-o", os.path.join(d, "s"), os.path.join(d, "s.c")], check=True)
        out = subprocess.run([os.path.join(d, "s")], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in out.split()] == [ctypes.sizeof(t) for t in (b.NormArgs, b.LinearFP8Args, b.GDNPrefillArgs)]


def test_the_binding_refuses_sizes_past_32_bits(monkeypatch):
    """Sizes that would arrive in the library cut to 32 bits (2^32 + 1 rows as one row, with no error)."""
    torch = pytest.importorskip("torch")
    b = rb()
    monkeypatch.setattr(b, "_on_device", lambda device, what="": device)
    monkeypatch.setattr(b, "_launch", lambda *a: pytest.fail("launched"))
    t = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    many, f32, e4m3 = (1 << 32) + 1, torch.float32, torch.float8_e4m3fn
    for x in (t(many, 8), t(1 << 31, 8), t(1, (1 << 32) + 128)):
        with pytest.raises(ValueError, match="2\\^31"):
            b.norm(x)
    for m, k, n in ((many, 128, 8), (1, 128, many), (2, (1 << 32) + 128, 8)):
        with pytest.raises(ValueError, match="2\\^31"):
            b.linear_fp8(t(m, k, dtype=e4m3), t(m, k // 128, dtype=f32), t(n, k, dtype=e4m3), t(-(-n // 128), k // 128, dtype=f32))
    for rows, H, dk, dv, starts in ((many, 1, 16, 16, 2), (4, 1, 16, 16, many), (1, many, 1, 1, 2), (1, 1, (1 << 32) + 16, 16, 2),
                                    (1, 1, 16, (1 << 32) + 16, 2)):
        args = (t(rows, H * dk), t(rows, H * dk), t(rows, H * dv), t(rows, H, dtype=f32), t(rows, H, dtype=f32),
                t(starts, dtype=torch.int32))
        with pytest.raises(ValueError, match="2\\^31"):
            b.gdn_prefill(*args)
        with pytest.raises(ValueError, match="2\\^31"):
            b.gdn_prefill_workspace(*args)
