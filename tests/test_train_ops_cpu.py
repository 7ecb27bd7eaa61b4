"""The training-side entry points on the host: sizes of workspaces, and every
refusal, which returns before anything would be launched."""
import ctypes

import pytest

import audio_video_flow_gb300 as h3
from audio_video_flow_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return h3.lib()


def _call(f, args, **changed):
    a = dict(args)
    a.update(changed)
    return f(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in a.values()])


ATTENTION = dict(n_rows=8, n_heads=4, q=0x1000, k=0x2000, v=0x3000, rs=512, hs=128, o=0x4000, d_o=0x5000, lse=0x6000,
                 dq=0x7000, dk=0x8000, dv=0x9000, drs=512, dhs=128, ws=0x10000, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("changed, status", [
    (dict(n_rows=0), h3.H3_ERR_SHAPE), (dict(n_rows=-1), h3.H3_ERR_SHAPE), (dict(n_heads=0), h3.H3_ERR_SHAPE),
    (dict(n_heads=65536), h3.H3_ERR_SHAPE), (dict(rs=120), h3.H3_ERR_SHAPE), (dict(hs=64), h3.H3_ERR_SHAPE),
    (dict(drs=0), h3.H3_ERR_SHAPE), (dict(dhs=-128), h3.H3_ERR_SHAPE), (dict(rs=513), h3.H3_ERR_ALIGN),
    (dict(hs=132), h3.H3_ERR_ALIGN), (dict(drs=516), h3.H3_ERR_ALIGN), (dict(dhs=129), h3.H3_ERR_ALIGN),
    (dict(q=0x1008), h3.H3_ERR_ALIGN), (dict(d_o=0x5002), h3.H3_ERR_ALIGN), (dict(dv=0x9008), h3.H3_ERR_ALIGN),
    (dict(lse=0x6002), h3.H3_ERR_ALIGN), (dict(ws=0x10010), h3.H3_ERR_ALIGN),
    (dict(dq=0x1000), h3.H3_ERR_SHAPE), (dict(dk=0x5000), h3.H3_ERR_SHAPE), (dict(dv=0x8000), h3.H3_ERR_SHAPE),
    (dict(ws_bytes=4095), h3.H3_ERR_WORKSPACE)])
def test_attention_backward_refuses(lib, changed, status):
    assert _call(lib.h3_attention_backward, ATTENTION, **changed) == status


@pytest.mark.parametrize("name", ["q", "k", "v", "o", "d_o", "lse", "dq", "dk", "dv", "ws"])
def test_attention_backward_refuses_null(lib, name):
    assert _call(lib.h3_attention_backward, ATTENTION, **{name: None}) == h3.H3_ERR_NULL


def test_attention_backward_workspace(lib):
    f = h3.h3_attention_backward_workspace_bytes
    assert f(1, 1) == 1024 and f(128, 1) == 1024 and f(129, 3) == 6 * 1024
    assert f(15860, 56) == 124 * 56 * 1024
    assert f(0, 1) == f(1, 0) == f(1, 65536) == f(-1, 1) == 0
    assert f(2 ** 31 - 1, 65535) == 2 ** 24 * 65535 * 1024       # past 32 bits


def _rope(**kw):
    base = dict(head_dim=128, n_axes=3, n_freqs=16)
    base.update(kw)
    return h3.make_rope_config(**base)


ROPE = dict(cfg=_rope(), n_rows=8, pos=0x100, direction=0, q_in=0x1000, q_out=0x2000, q_heads=4, k_in=0x3000,
            k_out=0x4000, k_heads=4, irs=512, ihs=128, ors=512, ohs=128, stream=None)


@pytest.mark.parametrize("changed, status", [
    (dict(n_rows=0), h3.H3_ERR_SHAPE), (dict(q_heads=0), h3.H3_ERR_SHAPE), (dict(k_heads=-1), h3.H3_ERR_SHAPE),
    (dict(q_heads=65536), h3.H3_ERR_SHAPE), (dict(direction=2), h3.H3_ERR_UNSUPPORTED),
    (dict(irs=120), h3.H3_ERR_SHAPE), (dict(ohs=120), h3.H3_ERR_SHAPE), (dict(irs=516), h3.H3_ERR_ALIGN),
    (dict(ohs=132), h3.H3_ERR_ALIGN), (dict(q_in=0x1008), h3.H3_ERR_ALIGN), (dict(k_out=0x4004), h3.H3_ERR_ALIGN),
    (dict(pos=0x102), h3.H3_ERR_ALIGN), (dict(pos=None), h3.H3_ERR_NULL), (dict(q_out=None), h3.H3_ERR_NULL),
    (dict(k_in=None), h3.H3_ERR_NULL),
    (dict(q_out=0x1000), h3.H3_ERR_SHAPE),                                # q in place, k not
    (dict(q_out=0x1000, k_out=0x3000, ors=640), h3.H3_ERR_SHAPE),         # in place with other strides
    (dict(q_out=0x1000, k_out=0x3000, ohs=136), h3.H3_ERR_SHAPE),
    (dict(k_out=0x2000), h3.H3_ERR_SHAPE), (dict(k_out=0x1000), h3.H3_ERR_SHAPE), (dict(q_out=0x3000), h3.H3_ERR_SHAPE),
    (dict(cfg=_rope(head_dim=127)), h3.H3_ERR_UNSUPPORTED), (dict(cfg=_rope(head_dim=0)), h3.H3_ERR_UNSUPPORTED),
    (dict(cfg=_rope(head_dim=258)), h3.H3_ERR_UNSUPPORTED), (dict(cfg=_rope(n_freqs=22)), h3.H3_ERR_UNSUPPORTED),
    (dict(cfg=_rope(n_axes=5, n_freqs=1)), h3.H3_ERR_UNSUPPORTED), (dict(cfg=_rope(n_axes=0)), h3.H3_ERR_UNSUPPORTED),
    (dict(cfg=_rope(n_freqs=0)), h3.H3_ERR_UNSUPPORTED), (dict(cfg=_rope(layout=2)), h3.H3_ERR_UNSUPPORTED),
    (dict(cfg=_rope(dtype=2)), h3.H3_ERR_UNSUPPORTED), (dict(cfg=_rope(scaling=4)), h3.H3_ERR_UNSUPPORTED),
    (dict(cfg=_rope(theta=1.0)), h3.H3_ERR_SHAPE), (dict(cfg=_rope(theta=float("nan"))), h3.H3_ERR_SHAPE),
    (dict(cfg=_rope(magnitude=0.0)), h3.H3_ERR_SHAPE), (dict(cfg=_rope(magnitude=float("inf"))), h3.H3_ERR_SHAPE),
    (dict(cfg=_rope(scaling=1, factor=0.5)), h3.H3_ERR_SHAPE),
    (dict(cfg=_rope(scaling=1, factor=2.0, scaled_axes=8)), h3.H3_ERR_SHAPE),
    (dict(cfg=_rope(scaling=2, n_freqs=1, factor=2.0)), h3.H3_ERR_UNSUPPORTED),
    (dict(cfg=_rope(scaling=3, factor=2.0, trained_length=0.0)), h3.H3_ERR_SHAPE),
    (dict(cfg=_rope(scaling=3, factor=2.0, alpha=32.0)), h3.H3_ERR_SHAPE),
    (dict(cfg=_rope(scaling=3, factor=2.0, alpha=-1.0)), h3.H3_ERR_SHAPE),
    (dict(cfg=None), h3.H3_ERR_NULL)])
def test_rope_refuses(lib, changed, status):
    assert _call(lib.h3_rope, ROPE, **changed) == status


def _norm(**kw):
    base = dict(kind=h3.H3_NORM_LAYER, width=128)
    base.update(kw)
    return h3.make_norm_config(**base)


FORWARD = dict(cfg=_norm(), n_rows=8, n_heads=4, x=0x1000, xrs=512, xhs=128, gain=0x2000, bias=0x3000, y=0x4000,
               yrs=512, yhs=128, stream=None)
BACKWARD = dict(cfg=_norm(), n_rows=8, n_heads=4, x=0x1000, xrs=512, xhs=128, gain=0x2000, dy=0x3000, dyrs=512,
                dyhs=128, dx=0x4000, dxrs=512, dxhs=128, dgain=0x5000, dbias=0x6000, ws=0x10000, ws_bytes=1 << 20,
                stream=None)
CONFIGS = [(dict(cfg=_norm(kind=2)), h3.H3_ERR_UNSUPPORTED), (dict(cfg=_norm(dtype=2)), h3.H3_ERR_UNSUPPORTED),
           (dict(cfg=_norm(param_dtype=-1)), h3.H3_ERR_UNSUPPORTED), (dict(cfg=_norm(width=0)), h3.H3_ERR_SHAPE),
           (dict(cfg=_norm(width=8193)), h3.H3_ERR_UNSUPPORTED), (dict(cfg=_norm(eps=0.0)), h3.H3_ERR_SHAPE),
           (dict(cfg=_norm(eps=float("nan"))), h3.H3_ERR_SHAPE), (dict(cfg=None), h3.H3_ERR_NULL),
           (dict(n_rows=0), h3.H3_ERR_SHAPE), (dict(n_heads=0), h3.H3_ERR_SHAPE), (dict(x=None), h3.H3_ERR_NULL),
           (dict(xrs=64), h3.H3_ERR_SHAPE), (dict(xhs=64), h3.H3_ERR_SHAPE), (dict(xrs=516), h3.H3_ERR_ALIGN),
           (dict(xhs=130), h3.H3_ERR_ALIGN), (dict(x=0x1008), h3.H3_ERR_ALIGN), (dict(gain=0x2008), h3.H3_ERR_ALIGN)]


@pytest.mark.parametrize("changed, status", CONFIGS + [
    (dict(y=None), h3.H3_ERR_NULL), (dict(yrs=516), h3.H3_ERR_ALIGN), (dict(yhs=64), h3.H3_ERR_SHAPE),
    (dict(y=0x4004), h3.H3_ERR_ALIGN), (dict(bias=0x3008), h3.H3_ERR_ALIGN),
    (dict(y=0x1000, yrs=640), h3.H3_ERR_SHAPE), (dict(y=0x1000, yhs=136), h3.H3_ERR_SHAPE)])
def test_norm_forward_refuses(lib, changed, status):
    assert _call(lib.h3_norm_forward, FORWARD, **changed) == status


@pytest.mark.parametrize("changed, status", CONFIGS + [
    (dict(dy=None), h3.H3_ERR_NULL), (dict(dx=None), h3.H3_ERR_NULL), (dict(ws=None), h3.H3_ERR_NULL),
    (dict(dyrs=516), h3.H3_ERR_ALIGN), (dict(dxhs=64), h3.H3_ERR_SHAPE), (dict(dx=0x4008), h3.H3_ERR_ALIGN),
    (dict(dgain=0x5002), h3.H3_ERR_ALIGN), (dict(dbias=0x6001), h3.H3_ERR_ALIGN), (dict(ws=0x10080), h3.H3_ERR_ALIGN),
    (dict(dx=0x3000, dxrs=640), h3.H3_ERR_SHAPE), (dict(dx=0x1000, dxhs=136), h3.H3_ERR_SHAPE),
    (dict(dgain=0x6000), h3.H3_ERR_SHAPE), (dict(ws_bytes=64), h3.H3_ERR_WORKSPACE),
    (dict(dgain=None, ws_bytes=0), h3.H3_ERR_WORKSPACE)])
def test_norm_backward_refuses(lib, changed, status):
    assert _call(lib.h3_norm_backward, BACKWARD, **changed) == status


def test_norm_workspace(lib):
    f = h3.h3_norm_backward_workspace_bytes
    assert f(_norm(width=5376), 1, 1) >= 2 * 5376 * 4
    assert f(_norm(width=5376), 505, 1) % 256 == 0
    assert f(_norm(width=8193), 8, 1) == 0 and f(_norm(), 0, 1) == 0 and f(_norm(), 1, 0) == 0
    # many rows: bounded by the GPU, not by the rows
    assert f(_norm(width=5376), 2 ** 31 - 1, 65535) <= 4096 * 2 * 5376 * 4


def test_binding_raises(lib):
    with pytest.raises(h3.H3Error) as e:
        h3.h3_norm_forward(_norm(width=8193), 1, 1, 0x1000, 8200, 8200, None, None, 0x9000, 8200, 8200, stream=0)
    assert e.value.status == h3.H3_ERR_UNSUPPORTED


@pytest.mark.parametrize("name, args, strides", [
    ("h3_attention_backward", ATTENTION, ("drs", "dhs")), ("h3_rope", ROPE, ("ors", "ohs")),
    ("h3_norm_forward", FORWARD, ("yrs", "yhs")), ("h3_norm_backward", BACKWARD, ("dxrs", "dxhs"))])
@pytest.mark.parametrize("row, head", [(128, 128), (256, 128), (504, 128), (128, 1016), (512, 136)])
def test_outputs_whose_rows_and_heads_overlap_are_refused(lib, name, args, strides, row, head):
    """8 rows of 4 heads of 128 channels."""
    assert _call(getattr(lib, name), args, **dict(zip(strides, (row, head)))) == h3.H3_ERR_SHAPE
