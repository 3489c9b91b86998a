"""The paged calls without a GPU: argument checks answer before any launch."""
import ctypes

import pytest

import temporally_compressed_latent_b200 as mtla

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def _space(n=1 << 16):
    # host memory stands in for device pointers: only argument checks run
    buf = (ctypes.c_uint8 * (n + 64))()
    return buf, (ctypes.addressof(buf) + 63) & ~63


KEEP, P = _space()


def _dims(**k):
    v = dict(H=8, d_h=64, r=256, d_R=32, s=2, dtype="bf16")
    v.update(k)
    return mtla.dims(*(v[x] for x in ("H", "d_h", "r", "d_R", "s", "dtype")))


def _chunk(N=4, start=P, prev=P, count=None):
    return mtla.chunk(N, start, prev, count)


def _cache(pages=P, num=10, rows=16, stride=288, table=P, entries=2):
    return mtla.paged_cache(pages, num, rows, stride, table, entries)


def _append(d=None, B=2, chunk=None, cache=None, base=1e4, q=P, qo=P, J=4, tail_in=P, tail_out=P + 8192, t_out=P + 4096,
            clen=None, state=P, err=P, c=P, merge=True):
    m = mtla.merge_args(c, P, P, P, P, J)
    return mtla.lib.mtla_paged_append(ctypes.byref(d or _dims()), B, ctypes.byref(chunk or _chunk()),
                                      ctypes.byref(m) if merge else None, base, q, qo, ctypes.byref(cache or _cache()),
                                      tail_in, tail_out, t_out, clen, state, None, 0, err, None)


def _attn(d=None, B=2, chunk=None, cache=None, qa=P, qr=P, state=P, out=P, od=1, lse=P, ws=P, size=0, err=P):
    return mtla.lib.mtla_paged_attn(ctypes.byref(d or _dims()), B, ctypes.byref(chunk or _chunk()), qa, qr, state,
                                    ctypes.byref(cache or _cache()), out, od, lse, ws, size, err, None)


@pytest.mark.parametrize("call", [_append, _attn], ids=["append", "attn"])
def test_shared_refusals(call):
    assert call(d=_dims(s=0)) == INVALID
    assert call(d=_dims(H=32)) == UNSUPPORTED
    assert call(d=_dims(r=252)) == UNSUPPORTED
    assert call(B=-1) == INVALID
    assert call(chunk=_chunk(N=-1)) == INVALID
    assert call(chunk=_chunk(start=None)) == INVALID
    assert call(chunk=_chunk(prev=None)) == INVALID
    assert call(chunk=_chunk(start=P + 2)) == INVALID
    assert call(chunk=_chunk(count=P + 1)) == INVALID
    assert call(chunk=_chunk(N=1 << 28)) == UNSUPPORTED     # N H rows
    assert call(cache=_cache(pages=None)) == INVALID
    assert call(cache=_cache(pages=P + 8)) == INVALID
    assert call(cache=_cache(table=None)) == INVALID
    assert call(cache=_cache(num=0)) == INVALID
    assert call(cache=_cache(entries=0)) == INVALID
    for rows in (0, 4, 12, -8):
        assert call(cache=_cache(rows=rows)) == INVALID
    assert call(cache=_cache(num=1 << 27, rows=16)) == INVALID   # 2^31 rows
    assert call(cache=_cache(stride=280)) == INVALID
    assert call(cache=_cache(stride=292)) == INVALID
    assert call(cache=_cache(stride=1 << 31)) == INVALID
    assert call(err=None) == INVALID


def test_append_refusals():
    assert _append(merge=False) == INVALID
    assert _append(c=None) == INVALID
    assert _append(c=P + 8) == INVALID
    assert _append(J=0) == INVALID
    assert _append(qo=None) == INVALID and _append(q=None) == INVALID
    assert _append(state=P + 2) == INVALID
    for base in (-1.0, float("inf"), float("nan")):
        assert _append(base=base) == INVALID
    assert _append(tail_in=None) == INVALID and _append(tail_out=None) == INVALID and _append(t_out=None) == INVALID
    # the state that is read is not overwritten
    assert _append(tail_out=P) == INVALID and _append(tail_out=P + 288 * 4) == INVALID
    assert _append(t_out=P + 4) == INVALID and _append(clen=P) == INVALID
    # no sequences: nothing to do
    assert _append(B=0, chunk=_chunk(N=0)) == 0
    assert _append(B=0, chunk=_chunk(N=0), c=None, q=None, qo=None, state=None) == 0


def test_attn_refusals():
    assert _attn(qa=None) == INVALID and _attn(qr=None) == INVALID and _attn(state=None) == INVALID
    assert _attn(out=None) == INVALID and _attn(out=P + 8) == INVALID and _attn(lse=P + 2) == INVALID
    assert _attn(od=2) == INVALID
    assert _attn(d=_dims(dtype="f32"), cache=_cache(), od=1) == INVALID
    assert _attn(B=0) == 0 and _attn(chunk=_chunk(N=0)) == 0
    assert _attn(chunk=_chunk(N=0), qa=None, qr=None, state=None, out=None, lse=None, ws=None) == 0


def test_verify_refusals():
    def call(B=1, N=3, V=10, p=P, ldp=10, q=P, ldq=10, tok=P, start=P, ua=P, us=P, keep=P, nxt=P, err=P):
        return mtla.lib.mtla_verify_drafts(B, N, V, p, ldp, q, ldq, tok, start, ua, us, keep, nxt, err, None)

    assert call(B=-1) == INVALID and call(N=-1) == INVALID and call(V=0) == INVALID and call(V=(1 << 22) + 1) == INVALID
    assert call(ldp=9) == INVALID and call(ldq=9) == INVALID
    for name in ("p", "tok", "start", "ua", "us", "keep", "nxt", "err"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: P + 2}) == INVALID
    assert call(B=0) == 0 and call(B=0, N=0, p=None, tok=None, ua=None) == 0


def test_workspace_query_needs_sound_arguments():
    assert mtla.mtla_paged_workspace_bytes(_dims(s=0), 1, 1, mtla.PAGED_ATTN) == 0
    assert mtla.mtla_paged_workspace_bytes(_dims(), 0, 1, mtla.PAGED_ATTN) == 0
    assert mtla.mtla_paged_workspace_bytes(_dims(), 1, 1, 9) == 0
    assert mtla.mtla_paged_workspace_bytes(_dims(), 1, 1, mtla.PAGED_APPEND) == 0


def test_binding_refuses_tensors_of_another_device():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("without a GPU there is no current device to compare with")
    with pytest.raises(Exception):
        mtla.mtla_verify_drafts(1, 3, 10, P, 10, P, 10, P, P, P, P, P, P, torch.zeros(1, dtype=torch.int32))


def test_binding_raises_on_error_status():
    with pytest.raises(mtla.MtlaError) as e:
        mtla.mtla_verify_drafts(1, 3, 0, P, 10, P, 10, P, P, P, P, P, P, P, stream=0)
    assert e.value.status == INVALID
    with pytest.raises(mtla.MtlaError) as e:
        mtla.mtla_paged_attn(_dims(), 2, _chunk(), P, P, P, _cache(rows=4), P, mtla.MTLA_BF16, None, P, 0, P, stream=0)
    assert e.value.status == INVALID
