"""Refusals of the paged cache's entry points on the host (no GPU): the C entries with addresses that are
never dereferenced, the Python bindings with tensors a kernel would misread."""
import glob
import os
import re

import pytest
import torch

from kv_cache_tempcache_gb300 import _lib as L

FAKE = 0x10000
I32MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    from kv_cache_tempcache_gb300 import build_lib
    build_lib.build()
    return L.load()


def append(lib, dtype=L.BF16, B=2, T=4, cu=FAKE, d=128, Hq=4, q=FAKE, qs=(512, 128), qo=FAKE + 4096, qos=(512, 128), Hk=2,
           k=FAKE, ks=(512, 128), v=FAKE, vs=(512, 128), wq=FAKE, wk=FAKE, eps=1e-6, axes=(44, 42, 42), pos=None,
           grid=(3, 4), theta=1e4, kp=FAKE, vp=FAKE + 16, pages=8, page=16, ps=(4096, 2048, 128), table=FAKE, max_pages=4,
           at=FAKE, ln=FAKE + 64):
    return lib.fastar_paged_append(dtype, B, T, cu, d, Hq, q, *qs, qo, *qos, Hk, k, *ks, v, *vs, wq, wk, eps, *axes, pos,
                                   *grid, theta, kp, vp, pages, page, *ps, table, max_pages, at, ln, None, None)


POOLS = [(dict(page=8), L.EINVAL), (dict(page=24), L.EINVAL), (dict(page=256), L.EINVAL), (dict(page=0), L.EINVAL),
         (dict(page=-16), L.EINVAL), (dict(pages=0), L.EINVAL), (dict(pages=2 ** 31), L.EINVAL), (dict(kp=None), L.EINVAL),
         (dict(vp=None), L.EINVAL), (dict(kp=FAKE + 8), L.EINVAL), (dict(vp=FAKE + 2), L.EINVAL), (dict(vp=FAKE), L.EINVAL),
         (dict(ps=(4096, 2048, 64)), L.EINVAL), (dict(ps=(64, 2048, 128)), L.EINVAL), (dict(ps=(4096, 64, 128)), L.EINVAL),
         (dict(ps=(4100, 2048, 128)), L.EINVAL), (dict(ps=(4096, 2052, 128)), L.EINVAL), (dict(ps=(4096, 2048, 132)), L.EINVAL),
         (dict(ps=(2 ** 38, 2048, 128)), L.EINVAL), (dict(B=0), L.EINVAL), (dict(B=65536), L.ECAPACITY), (dict(T=-1), L.EINVAL),
         (dict(T=2 ** 30 + 2), L.ECAPACITY), (dict(max_pages=0), L.EINVAL), (dict(max_pages=2 ** 26 + 1), L.ECAPACITY),
         (dict(max_pages=2 ** 62), L.ECAPACITY), (dict(table=None), L.EINVAL), (dict(at=None), L.EINVAL),
         (dict(cu=None, T=5), L.EINVAL), (dict(d=96), L.EUNSUPPORTED), (dict(dtype=2), L.EUNSUPPORTED)]


@pytest.mark.parametrize("kw,code", POOLS + [
    (dict(Hq=-1), L.EINVAL), (dict(Hk=0), L.EINVAL), (dict(axes=(43, 42, 42)), L.EINVAL), (dict(axes=(46, 42, 42)), L.EINVAL),
    (dict(axes=(-2, 0, 0)), L.EINVAL), (dict(theta=1.0), L.EINVAL), (dict(theta=float("nan")), L.EINVAL),
    (dict(eps=0.0), L.EINVAL), (dict(eps=float("inf")), L.EINVAL), (dict(grid=(0, 4)), L.EINVAL), (dict(wq=FAKE + 4), L.EINVAL),
    (dict(wk=FAKE + 8), L.EINVAL), (dict(k=None), L.EINVAL), (dict(v=FAKE + 4), L.EINVAL), (dict(ks=(512, 64)), L.EINVAL),
    (dict(vs=(512, 132)), L.EINVAL), (dict(qo=None), L.EINVAL), (dict(q=None), L.EINVAL), (dict(qs=(512, 100)), L.EINVAL),
    (dict(qo=FAKE, qos=(512, 256)), L.EINVAL), (dict(ln=FAKE), L.EINVAL), (dict(ln=FAKE + 4), L.EINVAL),
    (dict(ln=FAKE - 4), L.EINVAL), (dict(T=0, ln=None, k=None, v=None), L.OK)])
def test_append_refusals(lib, kw, code):
    assert append(lib, **kw) == code


@pytest.mark.parametrize("B", [2, 5])
def test_lengths_that_are_read_and_written_share_no_element(lib, B):
    far = dict(at=FAKE + 2 ** 20, cu=FAKE + 2 ** 21, table=FAKE + 2 ** 22, B=B, T=10, max_pages=3)
    for name, n in (("at", B), ("cu", B + 1), ("table", 3 * B)):
        for off in range(-4 * (B - 1), 4 * n, 4):
            assert append(lib, **dict(far, ln=far[name] + off)) == L.EINVAL, (name, off)


def attn(lib, q=FAKE, dtype=L.BF16, B=2, T=4, cu=FAKE, max_q=3, Hq=4, Hkv=2, d=128, qs=(512, 128), kp=FAKE, vp=FAKE + 16,
         pages=8, page=16, ps=(4096, 2048, 128), table=FAKE, max_pages=4, at=FAKE, block=0, window=0, sinks=0, scale=0.1,
         out=FAKE, os=(512, 128), ws=None, nb=0):
    return lib.fastar_paged_attn(q, dtype, B, T, cu, max_q, Hq, Hkv, d, *qs, kp, vp, pages, page, *ps, table, max_pages, at,
                                 block, window, sinks, scale, out, *os, None, None, ws, nb, None)


@pytest.mark.parametrize("kw,code", POOLS + [
    (dict(Hq=3), L.EINVAL), (dict(Hkv=0), L.EINVAL), (dict(Hq=-2), L.EINVAL), (dict(block=-1), L.EINVAL),
    (dict(window=-1), L.EINVAL), (dict(sinks=-1), L.EINVAL), (dict(scale=0.0), L.EINVAL), (dict(scale=-1.0), L.EINVAL),
    (dict(scale=float("nan")), L.EINVAL), (dict(scale=float("inf")), L.EINVAL), (dict(max_q=0), L.EINVAL),
    (dict(max_q=5), L.EINVAL), (dict(q=None), L.EINVAL), (dict(q=FAKE + 8), L.EINVAL), (dict(qs=(512, 4)), L.EINVAL),
    (dict(out=None), L.EINVAL), (dict(os=(512, 130)), L.EINVAL), (dict(T=2 ** 30), L.ECAPACITY),
    (dict(ws=FAKE + 8, nb=1000), L.EWORKSPACE), (dict(Hq=0), L.OK), (dict(T=0, q=None, out=None), L.OK)])
def test_attention_refusals(lib, kw, code):
    assert attn(lib, **kw) == code


def test_workspace(lib):
    w = lambda H=32, n=6, M=131072, d=128, B=8, r=1, P=6: L.workspace_bytes(L.OP_PAGED_ATTN, H, n, M, d, B, r=r, P=P)
    # one token each over long sequences: a slot a sequence and more, of all heads' outputs, maxima and sums
    assert w() >= 7 * 32 * 130 * 4
    assert w(M=100) == 0                                       # short sequences: keys are not split
    assert w(r=6, P=1, n=6000) > 0
    for bad in (dict(n=0), dict(M=0), dict(d=96), dict(B=0), dict(B=5), dict(r=0), dict(P=0), dict(n=2 ** 62), dict(n=2 ** 26),
                dict(r=7), dict(P=65536)):                      # the last: sizes that the call refuses
        assert w(**bad) == 0, bad
    assert w(M=2 ** 62) == w(M=2 ** 30)


def _args(H=2, T=4, d=128, pages=3, page=16, B=2, dtype=torch.bfloat16):
    pool = torch.zeros(2, pages, H, page, d, dtype=dtype)
    return dict(k=torch.zeros(H, T, d, dtype=dtype), v=torch.zeros(H, T, d, dtype=dtype), k_pool=pool[0], v_pool=pool[1],
                table=torch.zeros(B, 2, dtype=torch.int32), at=torch.zeros(B, dtype=torch.int32))


def test_bindings_refuse_other_shapes_types_and_devices(lib):
    def app(match, exc=ValueError, **kw):
        a = _args()
        a.update(kw)
        with pytest.raises(exc, match=match):
            L.fastar_paged_append(**a)

    good = _args()
    app("CUDA device")
    app("shape", v=good["v"][:, :3])
    app("unsupported", TypeError, k=good["k"].half())
    app("k_pool must be", k_pool=good["k_pool"].float())
    app("k_pool must have the shape", k_pool=good["k_pool"][:, :1])
    app("k_pool must have the shape", k_pool=good["k_pool"][..., :64])
    app("v_pool must have the shape", v_pool=good["v_pool"][0])
    app("share shape and strides", v_pool=good["v_pool"].transpose(1, 2).contiguous().transpose(1, 2))
    app("contiguous last", k_pool=good["k_pool"].transpose(2, 3).contiguous().transpose(2, 3))
    app("table must be", table=good["table"].long())
    app("two dimensions", table=good["table"][0])
    app("table must be contiguous", table=torch.zeros(2, 4, dtype=torch.int32)[:, ::2])
    app("at must have the shape", at=torch.zeros(3, dtype=torch.int32))
    app("cu must have the shape", cu=torch.zeros(2, dtype=torch.int32))
    app("len_out must be", len_out=torch.zeros(2))
    app("together", q=good["k"])
    app("q_out must have the shape", q=good["k"], q_out=good["k"][:1])
    app("wk must have the shape", wk=torch.zeros(64))
    app("pos must have the shape", pos=torch.zeros(4, 2, dtype=torch.int32))
    app("contiguous last", k=torch.zeros(2, 128, 4, dtype=torch.bfloat16).transpose(1, 2))

    def att(match, exc=ValueError, **kw):
        a = _args()
        a.pop("k"), a.pop("v")
        a.update(q=torch.zeros(4, 4, 128, dtype=torch.bfloat16), out=torch.zeros(4, 4, 128, dtype=torch.bfloat16), scale=0.1)
        a.update(kw)
        with pytest.raises(exc, match=match):
            L.fastar_paged_attn(**a)

    att("CUDA device")
    att("out must have the shape", out=torch.zeros(4, 5, 128, dtype=torch.bfloat16))
    att("out must be", out=torch.zeros(4, 4, 128))
    att("lse must have the shape", lse=torch.zeros(4, 5))
    att("v_pool must be", v_pool=good["v_pool"].float())
    att("dev_status must be", dev_status=torch.zeros(1))
    att("workspace must be contiguous", workspace=torch.zeros(64, 2)[:, 0])
    att("unsupported", TypeError, q=torch.zeros(4, 4, 128, dtype=torch.float16))


def test_packed_calls(lib):
    pack = lambda name, args: L._packer(0, name)[1](*args)
    a = [L.BF16, 2, 0, FAKE, 128, 0, 0, 512, 128, 0, 512, 128, 2, FAKE, 512, 128, FAKE, 512, 128, 0, 0, 1e-6, 44, 42, 42, 0, 3, 4,
         1e4, FAKE, FAKE + 16, 8, 16, 4096, 2048, 128, FAKE, 4, FAKE, 0, 0, 0]
    assert lib.fastar_packed_call(4, pack("fastar_paged_append", a), 42) == L.OK
    assert lib.fastar_packed_call(4, pack("fastar_paged_append", a), 41) == L.EINVAL
    a[28] = 0.5                                                # theta
    assert lib.fastar_packed_call(4, pack("fastar_paged_append", a), 42) == L.EINVAL
    b = [FAKE, L.BF16, 2, 0, FAKE, 0, 4, 2, 128, 512, 128, FAKE, FAKE + 16, 8, 16, 4096, 2048, 128, FAKE, 4, FAKE, 0, 0, 0, 0.1,
         FAKE, 512, 128, 0, 0, 0, 0, 0]
    assert lib.fastar_packed_call(5, pack("fastar_paged_attn", b), 33) == L.OK
    b[24] = -0.1
    assert lib.fastar_packed_call(5, pack("fastar_paged_attn", b), 33) == L.EINVAL
    b[24], b[6] = 0.1, 4 + 2 ** 32                             # an int that does not fit
    assert lib.fastar_packed_call(5, pack("fastar_paged_attn", b), 33) == L.EINVAL


def test_kernels_that_wait_for_the_one_before_make_no_promise_that_nothing_writes():
    from kv_cache_tempcache_gb300 import build_lib
    waiting = 0
    for path in glob.glob(os.path.join(build_lib.CSRC, "paged*.cu")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for kernel in text.split("__global__")[1:]:
            head, body = kernel.split("{", 1)
            assert "pdl_wait()" in body and "__restrict__" not in head, (path, head)
            waiting += 1
    assert waiting == 6                                       # append, three attentions, two joins


def test_no_block_leaves_before_it_has_waited_for_the_kernel_before():
    # where all blocks do, the launch is over before the one that it follows, and what comes next reads its outputs
    from kv_cache_tempcache_gb300 import build_lib
    for path in glob.glob(os.path.join(build_lib.CSRC, "*.cu")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for kernel in text.split("__global__")[1:]:
            first = kernel.find("pdl_wait()")
            assert first < 0 or not re.search(r"\breturn\b", kernel[:first]), (path, kernel[:200])


def test_most_tokens_of_a_call(lib):
    assert append(lib, T=2 ** 30) == attn(lib, T=2 ** 30, Hq=1, Hkv=1) == L.ECAPACITY
    assert attn(lib, T=2 ** 30 - 2, Hq=4) == L.ECAPACITY       # rows of all heads
    assert L.workspace_bytes(L.OP_PAGED_ATTN, 1, 2 ** 30, 100, 64, 1, r=1, P=1) == 0
    assert L.workspace_bytes(L.OP_PAGED_ATTN, 1, 2 ** 30 - 1, 100000, 64, 1, r=2 ** 30 - 1, P=1) > 0
