"""The upper limits of the sequence operators that include/dig_gla.h states: each is refused one
step beyond it, and passes the checks of the arguments at it (C entry points on fake addresses,
no GPU needed)."""
import pytest
import torch

from test_seq_refusals import fwd, lib, packed, rope, step  # noqa: F401

UNSUPPORTED = -2
FAR = [0x10000000 + (i << 52) for i in range(12)]   # apart enough for any size


def refused(rc):
    return rc == UNSUPPORTED


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses would be launched on")


def no_device():
    """The code the entry points give for good arguments here."""
    import gated_linear_attention_chunkwise_b200 as pkg
    return fwd(pkg.lib())


@needs_no_gpu
def test_limits_of_the_recurrence(lib):  # noqa: F811
    good = no_device()
    if good == UNSUPPORTED:
        pytest.skip("good arguments and limits are refused with the same code here")
    far = dict(x=FAR[1], gate=FAR[2], h0=FAR[3], out=FAR[4], last=FAR[5])
    assert fwd(lib, **far, B=1, C=65536, xs=65536, gs=65536) == good
    assert refused(fwd(lib, **far, B=1, C=65544, xs=65544, gs=65544))
    assert fwd(lib, **far, B=1 << 24) == good and refused(fwd(lib, **far, B=(1 << 24) + 1))
    assert fwd(lib, **far, B=1 << 20, Hg=1, Wg=1, C=4096, xs=4096, gs=4096) == good
    assert refused(fwd(lib, **far, B=(1 << 20) + 1, Hg=1, Wg=1, C=4096, xs=4096, gs=4096))
    assert fwd(lib, **far, B=1, Hg=1 << 15, Wg=1 << 15) == good
    assert refused(fwd(lib, **far, B=1, Hg=1 << 15, Wg=(1 << 15) + 1))
    assert fwd(lib, **far, xs=1 << 32) == good and refused(fwd(lib, **far, xs=(1 << 32) + 8))
    assert fwd(lib, **far, B=1, Hg=1, Wg=1 << 10, xs=1 << 32) == good
    assert refused(fwd(lib, **far, B=1, Hg=1, Wg=(1 << 10) + 1, xs=1 << 32))
    assert packed(lib, **far, cu=FAR[6], rows=1 << 30) == good
    assert refused(packed(lib, **far, cu=FAR[6], rows=(1 << 30) + 1))
    pool = dict(x=FAR[1], gate=FAR[2], st=FAR[3], so=FAR[3], slots=FAR[4], out=FAR[5])
    assert step(lib, **pool, N=65535, nslots=1 << 24) == good
    assert refused(step(lib, **pool, N=65536, nslots=1 << 24))
    assert refused(step(lib, **pool, nslots=(1 << 24) + 1))


@needs_no_gpu
def test_limits_of_the_rotation(lib):  # noqa: F811
    good = no_device()
    if good == UNSUPPORTED:
        pytest.skip("good arguments and limits are refused with the same code here")
    far = dict(q=FAR[1], k=FAR[2], pos=FAR[3], inv=FAR[4], qo=FAR[5], ko=FAR[6])
    wide = dict(Hq=4096, Hk=4096, qs=4096 * 64, ks=4096 * 64, qos=4096 * 64, kos=4096 * 64)
    assert rope(lib, **far, **wide) == good
    assert refused(rope(lib, **far, **{**wide, "Hq": 4097, "qs": 4097 * 64, "qos": 4097 * 64}))
    assert rope(lib, **far, rows=(1 << 31) // 6) == good and refused(rope(lib, **far, rows=(1 << 31) // 6 + 1))
    assert rope(lib, **far, qs=1 << 32) == good and refused(rope(lib, **far, qs=(1 << 32) + 8))
    assert rope(lib, **far, rows=1 << 10, qs=1 << 32) == good
    assert refused(rope(lib, **far, rows=(1 << 10) + 1, qs=1 << 32))
