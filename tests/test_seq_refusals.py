"""What the sequence operators refuse before anything is enqueued: the C entry points on
fake addresses that are never dereferenced, the binding on CPU tensors (no GPU needed)."""
import pytest
import torch

INVALID, UNSUPPORTED, ALIGN = -1, -2, -3
K = 0x100000


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._cuda_builder().build()
    import gated_linear_attention_chunkwise_b200 as pkg
    return pkg.lib()


def at(i):
    return 0x10000000 + i * K


def fwd(lib, x=at(1), gate=at(2), h0=at(3), B=2, Hg=4, Wg=4, C=64, xs=64, gs=64, d=0, norm=0.0, comp=0, dt=0, out=at(4),
        last=at(5)):
    return lib.glr_fwd(x, gate, h0, B, Hg, Wg, C, xs, gs, d, norm, comp, dt, out, last, None)


def packed(lib, x=at(1), gate=at(2), cu=at(6), h0=at(3), rows=32, n=3, C=64, xs=64, gs=64, d=0, norm=0.0, comp=0, dt=0,
           fill=0, out=at(4), last=at(5)):
    return lib.glr_fwd_packed(x, gate, cu, h0, rows, n, C, xs, gs, d, norm, comp, dt, fill, out, last, None)


def bwd(lib, x=at(1), gate=at(2), h=at(3), dout=at(4), h0=at(5), dl=at(6), B=2, Hg=4, Wg=4, C=64, xs=64, gs=64, d=0,
        norm=0.0, comp=0, dt=0, dx=at(7), dg=at(8), dh0=at(9)):
    return lib.glr_bwd(x, gate, h, dout, h0, dl, B, Hg, Wg, C, xs, gs, d, norm, comp, dt, dx, dg, dh0, None)


def step(lib, x=at(1), gate=at(2), st=at(3), slots=at(4), N=4, nslots=8, C=64, xs=64, gs=64, norm=0.0, comp=0, dt=0, fill=0,
         so=at(3), out=at(5)):
    return lib.glr_step(x, gate, st, slots, N, nslots, C, xs, gs, norm, comp, dt, fill, so, out, None)


def well_formed(rc):
    """Passed every check of the arguments: what is left is the device."""
    return rc in (0, -2, -4) if not torch.cuda.is_available() else True


@pytest.mark.parametrize("call", [fwd, packed, bwd])
def test_glr_shapes(lib, call):
    size = dict(rows=0) if call is packed else dict(Hg=0)
    assert call(lib, **size) == INVALID
    assert call(lib, C=0) == INVALID
    assert call(lib, d=12) == INVALID and call(lib, d=-1) == INVALID
    if call is packed:
        assert call(lib, d=2) == INVALID
        assert call(lib, cu=None) == INVALID
        assert call(lib, cu=at(6) + 2) == ALIGN
        assert call(lib, fill=2) == INVALID
        assert call(lib, n=0) == INVALID
        assert call(lib, rows=1 << 31) == UNSUPPORTED
    else:
        assert call(lib, B=0) == INVALID
        assert call(lib, Hg=1 << 16, Wg=1 << 16) == UNSUPPORTED
    assert call(lib, norm=-1.0) == INVALID and call(lib, norm=1e-31) == INVALID
    assert call(lib, norm=float("nan")) == INVALID and call(lib, norm=float("inf")) == INVALID
    assert call(lib, comp=2) == INVALID
    assert call(lib, dt=2) == INVALID
    assert call(lib, xs=56) == INVALID and call(lib, gs=60) == INVALID   # rows would overlap
    assert call(lib, C=60) == ALIGN                                      # 120-byte rows
    assert call(lib, xs=68) == ALIGN and call(lib, gs=66) == ALIGN
    assert call(lib, gs=66, norm=1.0) == ALIGN
    assert call(lib, C=65544, xs=65544, gs=65544) == UNSUPPORTED
    for name in ("x", "gate"):
        assert call(lib, **{name: None}) == INVALID
        assert call(lib, **{name: at(1) + 8}) == ALIGN


def test_glr_aliasing(lib):
    for call in (fwd, packed):
        assert call(lib, out=None) == INVALID
        for over in (at(1), at(2), at(3)):
            assert call(lib, out=over) == INVALID
        assert call(lib, out=at(1) - 16) == INVALID
        assert call(lib, last=at(4)) == INVALID
        assert call(lib, last=at(3) + 16) == INVALID      # h_last beside h0, not over it
        if not torch.cuda.is_available():
            assert well_formed(call(lib, last=at(3)))
            assert well_formed(call(lib, h0=None, last=None))
    assert packed(lib, out=at(6)) == INVALID
    for name in ("dx", "dg"):
        for over in range(1, 7):
            assert bwd(lib, **{name: at(over)}) == INVALID, (name, over)
        assert bwd(lib, **{name: None}) == INVALID
    assert bwd(lib, dx=at(8)) == INVALID
    assert bwd(lib, dh0=at(5)) == INVALID
    assert bwd(lib, h=None) == INVALID and bwd(lib, dout=None) == INVALID
    if not torch.cuda.is_available():
        assert well_formed(bwd(lib, dh0=at(6)))
        # out between the rows of a strided x would interleave: other pitch, refused; x and gate may
        assert well_formed(fwd(lib, gate=at(1) + 128, xs=128, gs=128, norm=1.0))


def test_step_refusals(lib):
    assert step(lib, N=0) == INVALID and step(lib, nslots=0) == INVALID
    assert step(lib, slots=None, N=9) == INVALID          # row 8 has no state
    assert step(lib, N=65536, nslots=1 << 17) == UNSUPPORTED
    assert step(lib, st=None) == INVALID and step(lib, so=None) == INVALID and step(lib, out=None) == INVALID
    assert step(lib, so=at(3) + 256) == INVALID           # neither in place nor apart
    assert step(lib, out=at(3)) == INVALID and step(lib, out=at(1)) == INVALID and step(lib, so=at(2)) == INVALID
    assert step(lib, slots=at(4) + 1) == ALIGN
    assert step(lib, x=at(1) + 4) == ALIGN and step(lib, C=12, xs=12, gs=12) == ALIGN
    assert step(lib, fill=-1) == INVALID and step(lib, norm=-2.0) == INVALID


def rope(lib, q=at(1), k=at(2), pos=at(3), p64=1, period=8, inv=at(4), rows=8, Hq=4, Hk=2, D=64, rot=64, qs=256, ks=128,
         inter=0, inverse=0, scale=1.0, dt=0, qo=at(5), qos=256, ko=at(6), kos=128):
    return lib.rope(q, k, pos, p64, period, inv, rows, Hq, Hk, D, rot, qs, ks, inter, inverse, scale, dt, qo, qos, ko, kos,
                    None)


def norm(lib, q=at(1), k=at(2), wq=at(7), wk=at(8), pos=at(3), p64=1, period=8, inv=at(4), rows=8, Hq=4, Hk=2, D=64, rot=64,
         qs=256, ks=128, inter=0, eps=1e-6, scale=1.0, dt=0, qo=at(5), qos=256, ko=at(6), kos=128):
    return lib.qk_norm_rope(q, k, wq, wk, pos, p64, period, inv, rows, Hq, Hk, D, rot, qs, ks, inter, eps, scale, dt, qo,
                            qos, ko, kos, None)


def norm_bwd(lib, gq=at(9), gk=at(10), q=at(1), k=at(2), wq=at(7), wk=at(8), pos=at(3), p64=1, period=8, inv=at(4), rows=8,
             Hq=4, Hk=2, D=64, rot=64, gqs=256, gks=128, qs=256, ks=128, inter=0, eps=1e-6, scale=1.0, dt=0, qo=at(5),
             qos=256, ko=at(6), kos=128, dwq=at(11), dwk=at(12)):
    return lib.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, p64, period, inv, rows, Hq, Hk, D, rot, gqs, gks, qs, ks, inter,
                                eps, scale, dt, qo, qos, ko, kos, dwq, dwk, None)


@pytest.mark.parametrize("call", [rope, norm, norm_bwd])
def test_heads_shapes(lib, call):
    assert call(lib, rows=0) == INVALID and call(lib, D=0) == INVALID and call(lib, Hq=0) == INVALID
    assert call(lib, Hk=-1) == INVALID
    assert call(lib, rot=72) == INVALID and call(lib, rot=-8) == INVALID
    assert call(lib, inv=None) == INVALID
    assert call(lib, pos=None, period=0) == INVALID
    assert call(lib, inter=2) == INVALID and call(lib, dt=5) == INVALID
    assert call(lib, scale=float("inf")) == INVALID and call(lib, scale=float("nan")) == INVALID
    assert call(lib, rot=36) == UNSUPPORTED and call(lib, D=60, rot=56) == UNSUPPORTED
    assert call(lib, D=264, rot=64, qs=4 * 264, ks=2 * 264) == UNSUPPORTED
    assert call(lib, rows=1 << 30) == UNSUPPORTED
    assert call(lib, qs=248) == INVALID and call(lib, qs=260) == ALIGN and call(lib, kos=132) == ALIGN
    assert call(lib, pos=at(3) + 4) == ALIGN
    for name in ("q", "k", "qo", "ko"):
        assert call(lib, **{name: None}) == INVALID
        assert call(lib, **{name: at(1) + 8}) == ALIGN
    # outputs over other inputs, over each other, or over an input with another stride
    assert call(lib, qo=at(2)) == INVALID and call(lib, ko=at(1)) == INVALID and call(lib, ko=at(5)) == INVALID
    assert call(lib, qo=at(1), qos=512) == INVALID
    assert call(lib, qo=at(3)) == INVALID and call(lib, ko=at(4)) == INVALID
    if not torch.cuda.is_available():
        # slices of one projection: q at column 0, k behind it
        pitch = dict(qs=512, ks=512, k=at(1) + 512)
        assert well_formed(call(lib, **pitch))
        assert well_formed(call(lib, Hk=0, k=None, ko=None))
        if call is not norm_bwd:
            assert well_formed(call(lib, **pitch, qo=at(1), qos=512, ko=at(1) + 512, kos=512))
            assert call(lib, **pitch, qo=at(1), qos=512, ko=at(1) + 496, kos=512) == INVALID
            assert well_formed(call(lib, pos=at(3) + 4, p64=0))


def test_norm_refusals(lib):
    for call in (norm, norm_bwd):
        assert call(lib, wq=None) == INVALID and call(lib, wk=None) == INVALID
        assert call(lib, eps=-1.0) == INVALID and call(lib, eps=float("nan")) == INVALID
        assert call(lib, wq=at(7) + 4) == ALIGN
    assert rope(lib, rot=0) == INVALID
    assert norm_bwd(lib, gq=None) == INVALID and norm_bwd(lib, dwk=None) == INVALID
    assert norm_bwd(lib, qo=at(1)) == INVALID            # not over the forward's input
    assert norm_bwd(lib, dwq=at(12)) == INVALID and norm_bwd(lib, dwq=at(5)) == INVALID
    if not torch.cuda.is_available():
        assert well_formed(norm(lib, rot=0, inv=None))
        assert well_formed(norm_bwd(lib, qo=at(9), ko=at(10)))


def test_binding_refuses_cpu_tensors_and_shapes():
    import gated_linear_attention_chunkwise_b200 as dig
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        dig.glr_fwd(x, x, 1, 4, 0)
    with pytest.raises(TypeError):
        dig.glr_fwd(x.half(), x, 1, 4, 0)
    with pytest.raises(TypeError):
        dig.glr_step(None, x, x)
    for norm in (0.0, -1.0, 1e-50, 1e39, float("nan")):   # 1e-50 would be 0 as fp32: log_alpha
        with pytest.raises(ValueError):
            dig.glr_fwd(x, x, 1, 4, 0, gate_norm=norm)
    with pytest.raises(TypeError):
        dig.rope(None, None, None, x)
    with pytest.raises(TypeError):
        dig.qk_norm_rope([1], None, None, None, None, x)
    with pytest.raises(ValueError):
        dig.rope(torch.zeros(3, 2, 8), None, None, torch.zeros(4))


def test_row_stride():
    from gated_linear_attention_chunkwise_b200 import _row_stride
    t = torch.zeros(3, 5, 32)
    assert _row_stride(t, "t", 2, 32) == 32
    assert _row_stride(t[..., 8:16], "t", 2, 8) == 32
    assert _row_stride(t[:1, :, :8], "t", 2, 8) == 32
    assert _row_stride(t[:, :1, :8], "t", 2, 8) == 160
    assert _row_stride(t[:1, :1, :8], "t", 2, 8) == 8
    assert _row_stride(torch.zeros(3, 5, 4, 8)[:, :, 1:3], "t", 2, 16) == 32
    for bad in (t[:, :4], t[..., ::2], t.transpose(0, 1), t.transpose(1, 2)):
        with pytest.raises(ValueError):
            _row_stride(bad, "t", 2, bad.shape[2])
