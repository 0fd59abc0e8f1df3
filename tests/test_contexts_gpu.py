"""The dense attend and the block insert after a device reset and in a second context of the device, though their shared
memory is asked for once a device.  In a child process, whose contexts are its own."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = r"""
import ctypes
import struct
import block_sparse_attention_03_gb300 as msa

lib = msa.lib()
rt, cu = ctypes.CDLL("libcudart.so.13"), ctypes.CDLL("libcuda.so.1")
rt.cudaMalloc.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
rt.cudaMemcpy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
rt.cudaMemset.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t]
ref = ctypes.byref
H, T, NB = 2, 300, 3


def ok(e):
    assert e == 0, e


def device(data=None, n=None):
    p = ctypes.c_void_p()
    ok(rt.cudaMalloc(ref(p), len(data) if data is not None else n))
    ok(rt.cudaMemset(p, 0, len(data) if data is not None else n))
    if data is not None:
        ok(rt.cudaMemcpy(p, data, len(data), 1))
    return p


def both():
    # 300 tokens whose K is 0 and V is 1, inserted (a CTA an item: more than 8 a span), and attended to
    ints = lambda *v: device(struct.pack("%di" % len(v), *v))
    table = ints(2, 0, 1)
    codes = H * 128 * 128 * NB
    c = msa.MsaCacheT(8, 0, NB, 128, H, 128, 128, device(n=codes), device(n=codes), None, None, device(n=4 * H * NB), device(n=4 * H * NB),
                      None, None, None, 0, 0, 0, 0)
    spans = msa.MsaSpansT(1, NB, ints(0), ints(T), ints(0), table)
    k, v = device(n=2 * T * H * 128), device(struct.pack("H", 0x3F80) * (T * H * 128))
    ws = device(n=256)
    got = [lib.msa_block_insert(ref(c), ref(spans), T, ref(msa.MsaRowsT(k, H * 128)), ref(msa.MsaRowsT(v, H * 128)), ws, 256, None)]
    b, f = msa.MsaBatchT(1, 1, NB, ints(T), table), msa.Config().struct()
    for heads in (H, 16 * H, 64 * H):  # one, two and two times four tiles of columns
        size = lib.msa_dense_workspace_size(ref(c), ref(b), heads)
        ws2, out = device(n=size), device(n=256 * heads)
        got.append(lib.msa_dense_attend(ref(c), ref(b), ref(f), ref(msa.MsaQueryT(device(n=256 * heads), 0, 1.0)), heads, out, None, ws2,
                                        size, None))
        ok(rt.cudaDeviceSynchronize())
        host = ctypes.create_string_buffer(256 * heads)
        ok(rt.cudaMemcpy(host, out, 256 * heads, 2))
        values = struct.unpack("%dH" % (128 * heads), host.raw)
        # V is 1 in 127 steps of 1 / 127, whose fp32 is not exact
        assert not any(got) and all(abs(x - 0x3F80) <= 1 for x in values), (got, set(values))
    return out


both()
ok(rt.cudaDeviceReset())
both()
ok(cu.cuInit(0))
ctx, of = ctypes.c_void_p(), ctypes.c_void_p()
ok(cu.cuCtxCreate_v2(ref(ctx), 0, 0))
ok(cu.cuPointerGetAttribute(ref(of), 1, both()))  # CU_POINTER_ATTRIBUTE_CONTEXT
assert of.value == ctx.value
both()
ok(cu.cuCtxDestroy_v2(ctx))
print("three contexts")
"""


def test_after_a_reset_and_in_a_second_context():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "three contexts" in r.stdout, (r.stdout, r.stderr)
