"""Refusals of the linear-attention operators: the C ABI's host checks (nothing is launched, so
they run without a GPU) and the binding's shape, type and stride checks."""
import ctypes
import os

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)          # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    from chunked_linear_recurrence_gb300 import _native
    if not os.path.exists(_native.LIB_PATH):
        from chunked_linear_recurrence_gb300 import build
        build.build()
    return _native.load()


def _shape(**kw):
    from chunked_linear_recurrence_gb300._native import sf_gdn_shape
    return ctypes.byref(sf_gdn_shape(**{**dict(B=1, T=64, H=1, K=128, V=128, N=1, dtype=1, scale=0.0), **kw}))


def _fwd(lib, shape, ptr=FAKE, decay=FAKE, cu=None, last=0, fin=None, ws=FAKE, ws_bytes=1 << 40):
    return lib.sf_linattn_chunk_fwd(shape, ptr, ptr, ptr, decay, None, cu, last, ptr, fin, ws, ws_bytes, None)


BAD = [(dict(K=96, V=96), 2), (dict(K=128, V=64), 2), (dict(T=-1), 1), (dict(H=0), 1), (dict(dtype=7), 1),
       (dict(N=2), 1), (dict(B=40000, T=40000, N=40000), 2), (dict(H=4, HK=3), 1), (dict(H=4, HK=-1), 1)]


@pytest.mark.parametrize("kw,status", BAD)
def test_chunked_entry_points_reject_bad_shapes(lib, kw, status):
    s = _shape(**kw)
    assert _fwd(lib, s) == status
    assert lib.sf_linattn_paged_chunk_fwd(s, FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, None, None, FAKE, FAKE,
                                          1 << 40, None) == status
    assert lib.sf_linattn_chunk_bwd(s, *([FAKE] * 4), None, None, FAKE, None, FAKE, FAKE, FAKE, None, FAKE,
                                    1 << 40, None) == status
    assert len(lib.sf_last_error()) > 0


def test_chunked_entry_points_reject_bad_pointers_and_workspaces(lib):
    s = _shape()
    assert _fwd(lib, s, ptr=None) == 1 and _fwd(lib, s, ptr=ODD) == 1 and _fwd(lib, s, decay=None) == 1
    assert _fwd(lib, s, last=1) == 1                                  # no final_state
    assert _fwd(lib, s, ws=None) == 3 and _fwd(lib, s, ws_bytes=8) == 3
    assert _fwd(lib, None) == 1
    assert _fwd(lib, _shape(B=2, N=3), cu=FAKE) == 1                  # cu_seqlens needs B == 1
    assert _fwd(lib, _shape(N=0), cu=FAKE) == 1
    paged = lambda **k: lib.sf_linattn_paged_chunk_fwd(               # noqa: E731
        s, FAKE, FAKE, FAKE, FAKE, k.get("cache", FAKE), k.get("slots", 4), k.get("idx", FAKE), None, None,
        FAKE, FAKE, 1 << 40, None)
    assert paged(cache=None) == 1 and paged(cache=ODD) == 1 and paged(slots=0) == 1 and paged(idx=None) == 1
    bwd = lambda do=FAKE, dq=FAKE, ws=1 << 40: lib.sf_linattn_chunk_bwd(   # noqa: E731
        s, *([FAKE] * 4), None, None, do, None, dq, FAKE, FAKE, None, FAKE, ws, None)
    assert bwd(do=None) == 1 and bwd(dq=None) == 1 and bwd(dq=ODD) == 1 and bwd(ws=64) == 3


def test_workspaces_that_are_not_16_byte_aligned_are_refused(lib):
    """The kernels read and write the segments' states in it 16 bytes at a time."""
    s = _shape(T=1 << 16)
    assert _fwd(lib, s, ws=ODD) == 3
    assert lib.sf_linattn_paged_chunk_fwd(s, FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, None, None, FAKE, ODD, 1 << 40,
                                          None) == 3
    assert lib.sf_linattn_chunk_bwd(s, *([FAKE] * 4), None, None, FAKE, None, FAKE, FAKE, FAKE, None, ODD,
                                    1 << 40, None) == 3
    assert lib.sf_qk_norm_rope_bwd(_qk(), *([FAKE] * 12), ODD, 1 << 40, None) == 3


def test_workspace_grows_with_segments_and_shared_heads(lib):
    """A walk of one segment needs the status word alone; a long one the states of its
    segments; grouped heads the per-value-head parts of dq and dk."""
    assert lib.sf_linattn_fwd_workspace(_shape(T=256), 0) == 256
    assert lib.sf_linattn_fwd_workspace(_shape(T=1 << 16), 0) > 256 + 2 * 65536
    plain = lib.sf_linattn_bwd_workspace(_shape(T=200, H=4), 0)
    grouped = lib.sf_linattn_bwd_workspace(_shape(T=200, H=4, HK=2), 0)
    assert grouped == plain + 2 * 200 * 4 * 128 * 4


def test_workspace_of_many_short_sequences(lib):
    """Only walks that are cut need entry states: T / seg whole segments and as many remainders at
    the most, whatever the number of sequences (a state of 32 heads is 2 MB; a forward's cut makes
    three pieces to a segment)."""
    state = 32 * 128 * 128 * 4
    fwd = lib.sf_linattn_fwd_workspace(_shape(T=65536, H=32, N=1024), 1)
    bwd = lib.sf_linattn_bwd_workspace(_shape(T=32768, H=32, N=512), 1)
    assert 256 < fwd <= 256 + 5 * 8 * state and 256 < bwd <= 256 + 3 * 5 * 8 * state


@pytest.mark.parametrize("delta", [False, True])
def test_steps_reject_bad_arguments(lib, delta):
    def call(shape, q=FAKE, gate=FAKE, cache=FAKE, slots=4, idx=FAKE, out=FAKE):
        if delta:
            return lib.sf_gdn_step(shape, q, FAKE, FAKE, gate, FAKE, cache, slots, idx, out, None)
        return lib.sf_linattn_step(shape, q, FAKE, FAKE, gate, cache, slots, idx, out, None)
    s = _shape(N=4)
    assert call(_shape(N=4, K=96, V=96)) == 2 and call(_shape(N=4, H=4, HK=3)) == 1
    assert call(_shape(N=-1)) == 1 and call(_shape(N=4, dtype=5)) == 1 and call(None) == 1
    assert call(s, q=None) == 1 and call(s, q=ODD) == 1 and call(s, cache=ODD) == 1 and call(s, out=None) == 1
    assert call(s, gate=None) == 1
    assert call(s, idx=None, slots=3) == 1                            # sequence 3 would have no slot
    assert call(_shape(N=1 << 30, H=4)) == 2
    assert call(_shape(N=0)) == 0                                     # nothing to do


def _qk(**kw):
    from chunked_linear_recurrence_gb300._native import sf_qk_shape
    d = dict(rows=4, H=4, HK=2, D=128, dtype=1, norm=0, eps=1e-6, rotary_dim=128, interleaved=0, table_rows=8,
             axes=1, rows_stride_q=512, rows_stride_k=256)
    sections = kw.pop("sections", (64,))
    d.update(kw)
    s = sf_qk_shape(**d)
    for a, n in enumerate(sections):
        s.sections[a] = n
    return ctypes.byref(s)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), 2), (dict(rotary_dim=132), 2), (dict(rotary_dim=12, sections=(6,)), 2), (dict(norm=2), 1),
    (dict(dtype=3), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(rows=-1), 1), (dict(H=0), 1),
    (dict(axes=0), 1), (dict(axes=5), 1), (dict(sections=(63,)), 1), (dict(axes=2, sections=(72, -8)), 1),
    (dict(table_rows=0), 1), (dict(rows_stride_q=508), 1), (dict(rows_stride_q=516), 1),
    (dict(rows_stride_k=128), 1)])
def test_norm_rope_rejects_bad_shapes(lib, kw, status):
    s = _qk(**kw)
    assert lib.sf_qk_norm_rope_fwd(s, *([FAKE] * 8), None) == status
    assert lib.sf_qk_norm_rope_bwd(s, *([FAKE] * 12), FAKE, 1 << 40, None) == status
    assert len(lib.sf_last_error()) > 0


def test_norm_rope_rejects_bad_pointers(lib):
    fwd = lambda s, q=FAKE, cs=FAKE, pos=FAKE, out=FAKE, w=FAKE: lib.sf_qk_norm_rope_fwd(   # noqa: E731
        s, q, FAKE, w, None, cs, pos, out, FAKE, None)
    s = _qk()
    assert fwd(s, q=None) == 1 and fwd(s, q=ODD) == 1 and fwd(s, cs=None) == 1 and fwd(s, pos=None) == 1
    assert fwd(s, out=None) == 1 and fwd(s, out=ODD) == 1 and fwd(s, w=ODD) == 1 and fwd(None) == 1
    assert lib.sf_qk_norm_rope_fwd(_qk(rows_stride_q=1024), FAKE, ctypes.c_void_p(1 << 21), None, None, FAKE,
                                   FAKE, FAKE, ctypes.c_void_p(1 << 22), None) == 1     # in place, strided
    assert fwd(_qk(rows=0)) == 0
    need = lib.sf_qk_norm_rope_bwd_workspace(s)
    bwd = lambda n: lib.sf_qk_norm_rope_bwd(s, *([FAKE] * 12), FAKE, n, None)   # noqa: E731
    assert bwd(need - 1) == 3


def test_binding_checks_shapes_types_and_strides():
    import chunked_linear_recurrence_gb300 as sf
    z = torch.zeros
    q, v, dec = z(1, 64, 2, 64), z(1, 64, 2, 64), z(2)
    with pytest.raises(ValueError, match="CUDA device"):
        sf.sf_linattn_chunk_fwd(q, q, v, dec)
    for kw, msg in ((dict(k=z(1, 64, 1, 64)), "k "), (dict(v=z(1, 32, 2, 64)), "does not match"),
                    (dict(v=v.bfloat16()), "one dtype"), (dict(decay=z(3)), "decay must be"),
                    (dict(cu_seqlens=z(2).long()), "int32")):
        a = {**dict(q=q, k=q, v=v, decay=dec), **kw}
        with pytest.raises(ValueError, match=msg):
            sf.sf_linattn_chunk_fwd(**a)
        with pytest.raises(ValueError, match=msg):
            sf.sf_linattn_chunk_bwd(initial_state=None, d_out=v, **a)
    with pytest.raises(ValueError, match="contiguous"):
        sf.sf_linattn_chunk_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), q, v, dec)
    t, c = z(3, 2, 64), z(4, 2, 64, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        sf.sf_linattn_step(t, t, t, dec, c)
    with pytest.raises(ValueError, match="state_cache"):
        sf.sf_linattn_step(t, t, t, dec, z(2, 64, 64))
    with pytest.raises(ValueError, match="q/k must be"):
        sf.sf_gdn_step(q, q, v, z(3, 2), z(3, 2), c)
    with pytest.raises(ValueError, match="norm must be"):
        sf.sf_qk_norm_rope_fwd(q, q, norm="layer")
    with pytest.raises(ValueError, match="one dtype"):
        sf.sf_qk_norm_rope_fwd(q, q.bfloat16())
    with pytest.raises(ValueError, match="CUDA device"):
        sf.sf_qk_norm_rope_fwd(q, q)


def test_no_query_heads_are_refused():
    """In the shape struct HK = 0 stands for H heads: a slice without any would be read as H."""
    import chunked_linear_recurrence_gb300 as sf
    z = torch.zeros
    q, v, dec, g = z(1, 64, 2, 64), z(1, 64, 2, 64), z(2), z(1, 64, 2)
    none, cache, idx = q[:, :, :0], z(4, 2, 64, 64), z(1, dtype=torch.int32)
    t = v[0]
    for call in (lambda: sf.sf_linattn_chunk_fwd(none, none, v, dec),
                 lambda: sf.sf_linattn_paged_chunk_fwd(none, none, v, dec, cache, idx),
                 lambda: sf.sf_linattn_chunk_bwd(none, none, v, dec, None, v),
                 lambda: sf.sf_linattn_fwd_workspace(none, v),
                 lambda: sf.sf_linattn_step(t[:, :0], t[:, :0], t, dec, cache),
                 lambda: sf.sf_gdn_step(t[:, :0], t[:, :0], t, z(64, 2), z(64, 2), cache),
                 lambda: sf.sf_gdn_chunk_fwd(none, none, v, g, g),
                 lambda: sf.sf_gdn_chunk_bwd(none, none, v, g, g, None, v)):
        with pytest.raises(ValueError, match="at least one head"):
            call()


def test_token_strides_of_a_fused_projection():
    from chunked_linear_recurrence_gb300._linattn import _token_stride
    x = torch.zeros(2, 5, (4 + 2 + 2) * 64)
    q = x[..., :256].view(2, 5, 4, 64)
    assert _token_stride("q", q) == 512
    assert _token_stride("q", q[:, :1]) == 5 * 512            # one token of each batch row
    assert _token_stride("q", q[:1, :1]) == 256               # one row: any stride does
    for bad in (q.transpose(1, 2), q[:, ::2], q[..., ::2], q[:, :4]):
        with pytest.raises(ValueError):
            _token_stride("q", bad)


def test_only_the_status_word_of_a_large_workspace_is_cleared(monkeypatch):
    from chunked_linear_recurrence_gb300 import _linattn
    monkeypatch.setattr(torch, "empty", lambda n, **kw: torch.full((n,), 255, **kw))
    n = (1 << 24) + 256
    ws = _linattn.workspace(n, "cpu")
    assert ws.numel() == n and not ws[:256].any() and (ws[256:] == 255).all()
    for n, size in ((8, 256), (4096, 4096), (1 << 24, 1 << 24)):
        ws = _linattn.workspace(n, "cpu")
        assert ws.numel() == size and not ws.any()


_NO_ENCODER_SCRIPT = r'''
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from chunked_linear_recurrence_gb300 import _native
lib = _native.load()
F, big, r = ctypes.c_void_p(1 << 20), 1 << 40, []
for D in (64, 128):
    s = ctypes.byref(_native.sf_gdn_shape(B=1, T=64, H=1, K=D, V=D, N=1, dtype=1, scale=0.0, HK=0))
    r.append((lib.sf_linattn_chunk_fwd(s, F, F, F, F, None, None, 0, F, None, F, big, None), lib.sf_last_error()))
    r.append((lib.sf_linattn_paged_chunk_fwd(s, F, F, F, F, F, 4, F, None, None, F, F, big, None),
              lib.sf_last_error()))
    r.append((lib.sf_linattn_chunk_bwd(s, F, F, F, F, None, None, F, None, F, F, F, None, F, big, None),
              lib.sf_last_error()))
print(repr(r))
'''


def test_bf16_without_tensor_map_encoder_is_unsupported(lib):
    """BF16 linear attention runs on the tensor-core kernel alone: with the driver's TMA descriptor
    encoder reported absent (in a child process) its entry points refuse and launch nothing."""
    import ast
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", _NO_ENCODER_SCRIPT, root], capture_output=True, text=True,
                         env=dict(os.environ, SF_GDN_DISABLE_TMA_ENCODER="1"), timeout=300)
    assert res.returncode == 0, res.stderr
    for status, msg in ast.literal_eval(res.stdout.strip().splitlines()[-1]):
        assert status == 2 and b"cuTensorMapEncodeTiled" in msg, (status, msg)
