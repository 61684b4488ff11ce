"""Refusals of the 4-bit cache's entry points and of the per-head norm and rotation, on the
host (no GPU): the C entries with addresses that are never dereferenced, the Python bindings
with tensors a kernel would misread."""
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


def rope(lib, dtype=L.BF16, n=4, d=128, Hq=2, q=FAKE, qs=(512, 128), qo=FAKE + 4096, qos=(512, 128), Hk=2,
         k=FAKE + 8192, ks=(512, 128), ko=FAKE + 16384, kos=(512, 128), wq=FAKE, wk=FAKE, eps=1e-6, axes=(44, 42, 42),
         pos=None, grid=(3, 4), theta=1e4):
    return lib.fastar_qk_norm_rope(dtype, n, d, Hq, q, *qs, qo, *qos, Hk, k, *ks, ko, *kos, wq, wk, eps, *axes, pos, 0,
                                   None, *grid, theta, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), L.EUNSUPPORTED), (dict(d=96), L.EUNSUPPORTED), (dict(d=256), L.EUNSUPPORTED),
    (dict(n=-1), L.EINVAL), (dict(n=2 ** 31), L.EINVAL), (dict(Hq=-1), L.EINVAL),
    (dict(axes=(43, 42, 42)), L.EINVAL), (dict(axes=(-2, 42, 42)), L.EINVAL), (dict(axes=(46, 42, 42)), L.EINVAL),
    (dict(theta=1.0), L.EINVAL), (dict(theta=float("inf")), L.EINVAL), (dict(theta=float("nan")), L.EINVAL),
    (dict(eps=0.0), L.EINVAL), (dict(eps=float("nan")), L.EINVAL), (dict(grid=(0, 4)), L.EINVAL),
    (dict(q=None), L.EINVAL), (dict(q=FAKE + 8), L.EINVAL), (dict(qs=(512, 120)), L.EINVAL),
    (dict(qs=(512, 132)), L.EINVAL), (dict(qo=None), L.EINVAL), (dict(k=None), L.EINVAL), (dict(ko=FAKE + 2), L.EINVAL),
    (dict(wq=FAKE + 4), L.EINVAL), (dict(wk=FAKE + 8), L.EINVAL),
    (dict(qo=FAKE, qos=(512, 256)), L.EINVAL),                                  # in place with other strides
    (dict(n=0, q=None, qo=None, k=None, ko=None), L.OK), (dict(Hq=0, Hk=0), L.OK)])
def test_norm_rope_refusals(lib, kw, code):
    assert rope(lib, **kw) == code


def append(lib, dtype=L.BF16, H=2, n=4, d=128, k=FAKE, ks=(512, 128), v=FAKE, vs=(512, 128), at=FAKE, kc=FAKE,
           ksc=FAKE + 16, vc=FAKE + 32, vsc=FAKE + 48, cap=64, len_out=FAKE + 64):
    return lib.fastar_kv4_append(dtype, H, n, d, k, *ks, v, *vs, None, None, at, kc, ksc, vc, vsc, cap, len_out, None,
                                 None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), L.EUNSUPPORTED), (dict(d=32), L.EUNSUPPORTED), (dict(H=-1), L.EINVAL), (dict(n=-1), L.EINVAL),
    (dict(cap=0), L.EINVAL), (dict(cap=60), L.EINVAL), (dict(cap=2 ** 31), L.EINVAL), (dict(n=65), L.ECAPACITY),
    (dict(len_out=FAKE), L.EINVAL), (dict(k=None), L.EINVAL), (dict(v=FAKE + 4), L.EINVAL),
    (dict(vs=(512, 64)), L.EINVAL), (dict(kc=None), L.EINVAL), (dict(ksc=FAKE + 8), L.EINVAL),
    (dict(vc=FAKE), L.EINVAL), (dict(vsc=FAKE + 16), L.EINVAL), (dict(H=0, k=None, v=None), L.OK),
    (dict(n=0, len_out=None, k=None), L.OK)])
def test_append_refusals(lib, kw, code):
    assert append(lib, **kw) == code


def read(lib, dtype=L.BF16, H=2, n=4, d=128, codes=FAKE, scales=FAKE, cap=64, first=0, out=FAKE, os=(512, 128)):
    return lib.fastar_kv4_read(dtype, H, n, d, codes, scales, None, cap, first, out, *os, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), L.EUNSUPPORTED), (dict(d=16), L.EUNSUPPORTED), (dict(first=-1), L.EINVAL),
    (dict(first=61), L.ECAPACITY), (dict(n=65), L.ECAPACITY), (dict(first=2 ** 62, n=2 ** 62), L.ECAPACITY),
    (dict(cap=72), L.EINVAL), (dict(codes=None), L.EINVAL), (dict(scales=FAKE + 1), L.EINVAL),
    (dict(out=None), L.EINVAL), (dict(os=(512, 100)), L.EINVAL), (dict(n=0, out=None), L.OK),
    (dict(first=64, n=0), L.OK)])
def test_read_refusals(lib, kw, code):
    assert read(lib, **kw) == code


def attn(lib, q=FAKE, dtype=L.BF16, Hq=4, Hkv=2, nq=4, d=128, qs=(512, 128), kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE,
         cap=64, len=FAKE, block=0, scale=0.1, out=FAKE, os=(512, 128), ws=None, nb=0):
    return lib.fastar_kv4_attn(q, dtype, Hq, Hkv, nq, d, *qs, kc, ks, vc, vs, None, None, cap, len, block, scale, out,
                               *os, None, None, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), L.EUNSUPPORTED), (dict(d=80), L.EUNSUPPORTED), (dict(Hq=3), L.EINVAL), (dict(Hkv=0), L.EINVAL),
    (dict(nq=-1), L.EINVAL), (dict(block=-1), L.EINVAL), (dict(cap=65), L.EINVAL), (dict(scale=0.0), L.EINVAL),
    (dict(scale=-1.0), L.EINVAL), (dict(scale=float("nan")), L.EINVAL), (dict(scale=float("inf")), L.EINVAL),
    (dict(nq=I32MAX), L.ECAPACITY), (dict(q=None), L.EINVAL), (dict(q=FAKE + 8), L.EINVAL),
    (dict(qs=(512, 4)), L.EINVAL), (dict(out=None), L.EINVAL), (dict(kc=None), L.EINVAL), (dict(vs=FAKE + 4), L.EINVAL),
    (dict(len=None), L.EINVAL), (dict(cap=65536, ws=FAKE, nb=16), L.EWORKSPACE), (dict(Hq=0), L.OK),
    (dict(nq=0, q=None, out=None), L.OK)])
def test_attention_refusals(lib, kw, code):
    assert attn(lib, **kw) == code


def test_workspace(lib):
    # one token over a long cache: partial outputs, maxima and sums of at least two splits
    assert L.workspace_bytes(L.OP_KV4_ATTN, 32, 1, 131072, 128, 8) >= 2 * 32 * 130 * 4
    for bad in (dict(n=0), dict(M=0), dict(d=96), dict(B=0), dict(B=5), dict(n=2 ** 62), dict(n=2 ** 26),
                dict(M=2 ** 62)):                          # the last three: sizes that the call refuses
        a = dict(H=32, n=1, M=131072, d=128, B=8)
        a.update(bad)
        assert L.workspace_bytes(L.OP_KV4_ATTN, a["H"], a["n"], a["M"], a["d"], a["B"]) == 0


def _cache(H=2, cap=64, d=128):
    return (torch.zeros(H, cap, d // 2, dtype=torch.uint8), torch.zeros(H, cap, d // 16, dtype=torch.uint8)) * 2


def _rows(H=2, n=4, d=128, dtype=torch.bfloat16):
    return torch.zeros(H, n, d, dtype=dtype)


def test_bindings_refuse_other_shapes_types_and_devices(lib):
    k, c = _rows(), _cache()
    i2 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        L.fastar_kv4_append(k, k, *c)
    with pytest.raises(ValueError, match="shape"):
        L.fastar_kv4_append(k, _rows(n=3), *c)
    with pytest.raises(TypeError):
        L.fastar_kv4_append(_rows(dtype=torch.float16), k, *c)
    with pytest.raises(ValueError, match="shape"):
        L.fastar_kv4_read(c[0], c[1][:, :, :4], 0, k)
    with pytest.raises(ValueError, match="must be torch.uint8"):
        L.fastar_kv4_read(c[0].to(torch.int8), c[1], 0, k)
    with pytest.raises(ValueError, match="contiguous"):
        L.fastar_kv4_read(c[0].transpose(0, 1).contiguous().transpose(0, 1), c[1], 0, k)
    with pytest.raises(ValueError, match="shape"):
        L.fastar_kv4_attn(k, *c, i2, 0.1, _rows(n=5))
    with pytest.raises(ValueError, match="contiguous last"):
        L.fastar_kv4_attn(_rows(2, 128, 4).transpose(1, 2), *c, i2, 0.1, k)
    with pytest.raises(ValueError, match="together"):
        L.fastar_qk_norm_rope(k, k, k, None)
    with pytest.raises(ValueError, match="shape"):
        L.fastar_qk_norm_rope(k, k, k, _rows(n=5))


def test_packed_calls(lib):
    # the arguments as 64-bit words: refused like the calls themselves, and by their own number and range
    def words(name, args):
        return L._packer(0, name)[1](*args)

    read = [L.BF16, 2, 4, 128, FAKE, FAKE, 0, 64, 0, FAKE, 512, 128, 0]
    for change, code in (({2: 0}, L.OK), ({7: 65}, L.EINVAL), ({0: 7}, L.EUNSUPPORTED), ({8: 61}, L.ECAPACITY),
                         ({1: 2 ** 31}, L.EINVAL), ({3: 128 + 2 ** 32}, L.EINVAL), ({4: 0}, L.EINVAL)):
        a = list(read)
        for i, v in change.items():
            a[i] = v
        assert lib.fastar_packed_call(2, words("fastar_kv4_read", a), 13) == code, change
    good = words("fastar_kv4_read", read[:2] + [0] + read[3:])
    assert lib.fastar_packed_call(2, good, 13) == L.OK
    for call, w, n in ((2, good, 12), (2, good, 14), (4, good, 13), (-1, good, 13), (2, None, 13)):
        assert lib.fastar_packed_call(call, w, n) == L.EINVAL
    # a float travels as a double's bits: the scale of the attention, the base of the rotation
    attn = [FAKE, L.BF16, 2, 2, 0, 128, 512, 128, FAKE, FAKE, FAKE, FAKE, 0, 0, 64, FAKE, 0, 0.1, FAKE, 512, 128, 0, 0,
            0, 0, 0]
    assert lib.fastar_packed_call(3, words("fastar_kv4_attn", attn), 26) == L.OK
    attn[17] = -0.1
    assert lib.fastar_packed_call(3, words("fastar_kv4_attn", attn), 26) == L.EINVAL
    rope_args = [L.BF16, 0, 128, 2, FAKE, 512, 128, FAKE, 512, 128, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1e-6, 44, 42, 42, 0, 0, 0, 3,
                 4, 1e4, 0]
    assert lib.fastar_packed_call(0, words("fastar_qk_norm_rope", rope_args), 30) == L.OK
    rope_args[28] = 0.5
    assert lib.fastar_packed_call(0, words("fastar_qk_norm_rope", rope_args), 30) == L.EINVAL


def test_kernels_that_wait_for_the_one_before_make_no_promise_that_nothing_writes():
    """A kernel launched while its predecessor still writes must not take that memory as __restrict__: the
    compiler may then load it before the wait.  The 4-bit cache's kernels and the norm's."""
    import glob
    import os
    import re
    from kv_cache_tempcache_gb300 import build_lib
    waiting = 0
    for path in glob.glob(os.path.join(build_lib.CSRC, "kv4*.cu")) + [os.path.join(build_lib.CSRC, "qk_rope.cu")]:
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for kernel in text.split("__global__")[1:]:
            head, body = kernel.split("{", 1)
            if "pdl_wait()" in body.split("__global__")[0]:
                waiting += 1
                assert "__restrict__" not in head, (path, head)
    assert waiting == 6                                     # norm, append, read, the two attentions, the join


@pytest.mark.parametrize("H", [2, 5])
def test_lengths_that_are_read_and_written_share_no_element(lib, H):
    for off in range(-4 * (H - 1), 4 * H, 4):
        assert append(lib, H=H, at=FAKE + 256, len_out=FAKE + 256 + off) == L.EINVAL, off
