"""Refusals of the paged cache's calls and of the few tokens' experts, on the host: the C entry points return their
status before any device work, and the wrappers raise before they call them.  Stand-in addresses: on machines without
a GPU only, where nothing could be launched on them."""
import ctypes
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="stand-in addresses: needs a machine without a GPU")

FAKE = 1 << 20
OK, ARG, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 7
PAST = (4, 5)  # checks passed: no device


@pytest.fixture(scope="module")
def nv():
    import nvfp4_bit_precision_b200 as nv
    return nv


CACHE = dict(q=FAKE, sf=FAKE, amax=FAKE, pages=8, kv_heads=2, page_size=16, dim=128)


def view(nv, kw):
    c = dict(CACHE)
    for name in list(kw):
        if name.startswith("c_"):
            c[name[2:]] = kw.pop(name)
    return nv.KVCacheView(*c.values())


def append(nv, **kw):
    c = view(nv, kw)
    a = dict(k=FAKE, ldk=1024, hsk=128, v=FAKE, ldv=1024, hsv=128, tokens=3, table=FAKE, ldt=4, sequences=3, pages=4, position=FAKE,
             sequence=None, cos=FAKE, sin=FAKE, angles=64, rot=128, neighbours=0, q=FAKE, ldq=1024, hsq=128, heads=4, qo=FAKE, ldo=512,
             hso=128, ws=None, n=0)
    a.update(kw)
    return nv._lib.nvfp4_kv_append(ctypes.byref(c), *a.values(), None)


BAD_CACHES = [
    (dict(c_q=None), ARG), (dict(c_sf=None), ARG), (dict(c_amax=None), ARG), (dict(c_pages=0), SHAPE), (dict(c_pages=1 << 31), SHAPE),
    (dict(c_kv_heads=0), SHAPE), (dict(c_page_size=8), SHAPE), (dict(c_page_size=48), SHAPE), (dict(c_page_size=2048), SHAPE),
    (dict(c_dim=96), SHAPE), (dict(c_dim=512), SHAPE), (dict(c_q=FAKE + 8), ALIGN), (dict(c_sf=FAKE + 4), ALIGN), (dict(c_amax=FAKE + 2), ALIGN)]


@pytest.mark.parametrize("change,status", BAD_CACHES + [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(table=None), ARG), (dict(position=None), ARG), (dict(sin=None), ARG), (dict(cos=None), ARG),
    (dict(q=None), ARG), (dict(qo=None), ARG), (dict(heads=0), ARG), (dict(cos=None, sin=None, rot=0), ARG), (dict(neighbours=2), ARG),
    (dict(pages=0, ldt=0), ARG), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(sequences=2), SHAPE), (dict(ldt=3), SHAPE),
    (dict(rot=16), SHAPE), (dict(rot=48), SHAPE), (dict(rot=160), SHAPE), (dict(rot=0), SHAPE), (dict(hsk=64), SHAPE), (dict(hsv=64), SHAPE),
    (dict(hsq=64), SHAPE), (dict(hso=64), SHAPE), (dict(ldo=64), SHAPE), (dict(angles=-1), SHAPE), (dict(ldk=-8), SHAPE),
    (dict(k=FAKE + 8), ALIGN), (dict(ldk=1028), ALIGN), (dict(hsk=132), ALIGN), (dict(v=FAKE + 2), ALIGN), (dict(ldv=1028), ALIGN),
    (dict(q=FAKE + 8), ALIGN), (dict(ldq=1028), ALIGN), (dict(qo=FAKE + 8), ALIGN), (dict(hso=132), ALIGN), (dict(cos=FAKE + 4), ALIGN),
    (dict(table=FAKE + 2), ALIGN), (dict(position=FAKE + 1), ALIGN), (dict(sequence=FAKE + 2), ALIGN), (dict(ws=FAKE, n=8), WORKSPACE),
    (dict(ws=FAKE + 8, n=256), WORKSPACE)])
def test_append_argument_errors(nv, change, status):
    assert append(nv, **change) == status


def test_append_refuses_heads_that_overlap(nv):
    """Turned queries are written: each head has its own place, token by token or head by head."""
    for ldo, hso, status in ((128, 128, SHAPE), (256, 128, SHAPE), (504, 128, SHAPE), (128, 256, SHAPE), (128, 376, SHAPE), (512, 128, PAST),
                             (128, 384, PAST), (1024, 136, PAST), (512, 136, SHAPE), (1 << 40, 1 << 20, PAST), (1 << 62, 1 << 62, SHAPE)):
        assert append(nv, ldo=ldo, hso=hso) in (status if status is PAST else (status,)), (ldo, hso)
    assert append(nv, ldo=0, hso=128, tokens=1) in PAST and append(nv, ldo=128, hso=0, heads=1) in PAST


def test_append_accepts(nv):
    for change in (dict(), dict(sequence=FAKE, sequences=1), dict(q=None, qo=None, heads=0), dict(q=None, qo=None, heads=0, cos=None, sin=None, rot=0),
                   dict(rot=32), dict(ws=FAKE, n=16), dict(ldk=0), dict(c_kv_heads=1, hsk=0, hsv=0)):
        assert append(nv, **change) in PAST


def test_append_accepts_no_tokens(nv):
    """Tensors without a token have no address, those of the queries among them."""
    none = dict(tokens=0, k=None, v=None, position=None, q=None, qo=None)
    for change in (none, dict(none, heads=0), dict(none, heads=0, cos=None, sin=None, rot=0), dict(none, sequence=None, sequences=0, table=None)):
        assert append(nv, **change) in PAST


def attend(nv, **kw):
    c = view(nv, kw)
    a = dict(q=FAKE, ldb=1024, ldi=512, ldh=128, sequences=3, queries=2, heads=4)
    b = dict(table=FAKE, ldt=4, pages=4, lengths=FAKE, scale=0.1, window=0, out=FAKE, lse=FAKE, ws=FAKE, n=1 << 30)
    a.update({k: kw.pop(k) for k in list(kw) if k in a})
    b.update(kw)
    return nv._lib.nvfp4_kv_attention(*a.values(), ctypes.byref(c), *b.values(), None)


@pytest.mark.parametrize("change,status", BAD_CACHES + [
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(lengths=None), ARG), (dict(table=None), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(heads=3), SHAPE), (dict(heads=0), SHAPE), (dict(queries=0), SHAPE), (dict(queries=(1 << 20) + 1), SHAPE),
    (dict(sequences=-1), SHAPE), (dict(sequences=(1 << 20) + 1), SHAPE), (dict(ldt=3), SHAPE), (dict(pages=-1, ldt=0), SHAPE), (dict(window=-1), SHAPE),
    (dict(ldh=64), SHAPE), (dict(ldb=-8), SHAPE), (dict(ldi=-8), SHAPE), (dict(pages=1 << 27, ldt=1 << 27), SHAPE),
    (dict(pages=1 << 20, ldt=1 << 20, sequences=1 << 18), SHAPE), (dict(q=FAKE + 8), ALIGN), (dict(ldi=516), ALIGN), (dict(ldb=1028), ALIGN),
    (dict(ldh=132), ALIGN), (dict(out=FAKE + 8), ALIGN), (dict(lse=FAKE + 2), ALIGN), (dict(table=FAKE + 2), ALIGN), (dict(lengths=FAKE + 1), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 8), WORKSPACE), (dict(n=128), WORKSPACE)])
def test_attention_argument_errors(nv, change, status):
    assert attend(nv, **change) == status


def test_attention_accepts(nv):
    for change in (dict(), dict(lse=None), dict(window=5), dict(scale=-1.0), dict(table=None, pages=0, ldt=0), dict(heads=128, ldi=16384, ldb=32768),
                   dict(c_dim=256, ldh=256), dict(sequences=1 << 20), dict(pages=1 << 20, ldt=1 << 20)):
        assert attend(nv, **change) in PAST


def test_attention_workspace(nv):
    size = nv.nvfp4_kv_attention_workspace_size
    assert size(0, 1, 8, 8, 128, 100) == size(1, 0, 8, 8, 128, 100) == size(1, 1, 4, 8, 128, 100) == size(1, 1, 8, 8, 96, 100) == 256
    assert 256 < size(1, 1, 8, 8, 128, 0) <= size(1, 1, 8, 8, 128, 100) <= size(1, 1, 32, 8, 128, 10000) <= size(64, 1, 32, 8, 128, 10000) < 1 << 26
    assert size(1 << 20, 1 << 10, 64, 1, 256, 1 << 31) < 1 << 26


@pytest.mark.parametrize("sizes", [(1, 65536, 65536, 1, 128, 100), (4, 1 << 20, 65536, 1, 64, 4096), (1, 65536, 32768, 1, 64, 100),
                                   (64, 1 << 20, 65536, 3, 64, 100), (1 << 20, 1 << 20, 65536, 65536, 64, 1 << 31), (1, 1, 8, 8, 128, 1 << 62),
                                   ((1 << 20) + 1, 1, 8, 8, 128, 100)])
def test_attention_workspace_of_sizes_that_are_refused(sizes):
    """Products of sizes past 31 and 64 bits: the status word's bytes, in a process of its own, which must not end."""
    call = f"import nvfp4_bit_precision_b200 as nv; print(nv.nvfp4_kv_attention_workspace_size{sizes})"
    done = subprocess.run([sys.executable, "-c", call], capture_output=True, text=True, timeout=120)
    assert done.returncode == 0 and done.stdout.strip() == "256", (done.returncode, done.stdout)


def mlp(nv, **kw):
    a = dict(G=4, off=FAKE, rows=8, x=FAKE, ldx=256, tokens=4, index=FAKE, gq=FAKE, gs=FAKE, gg=FAKE, uq=FAKE, us=FAKE, ug=FAKE, dq=FAKE, ds=FAKE,
             dg=FAKE, hidden=256, ffn=128, slot=FAKE, weight=FAKE, k=2, base=FAKE, out=FAKE, ws=FAKE, n=1 << 20)
    a.update(kw)
    return nv._lib.nvfp4_expert_mlp(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(G=0), ARG), (dict(G=257), ARG), (dict(off=None), ARG), (dict(x=None), ARG), (dict(index=None), ARG), (dict(gq=None), ARG), (dict(gs=None), ARG),
    (dict(gg=None), ARG), (dict(uq=None), ARG), (dict(us=None), ARG), (dict(ug=None), ARG), (dict(dq=None), ARG), (dict(ds=None), ARG),
    (dict(dg=None), ARG), (dict(slot=None), ARG), (dict(weight=None), ARG), (dict(out=None), ARG), (dict(hidden=192), SHAPE), (dict(ffn=64), SHAPE),
    (dict(hidden=0), SHAPE), (dict(ffn=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE),
    (dict(ldx=128), SHAPE), (dict(hidden=1 << 17, ldx=1 << 17), SHAPE), (dict(ffn=1 << 17, n=1 << 40), SHAPE), (dict(x=FAKE + 8), ALIGN),
    (dict(ldx=260), ALIGN), (dict(gq=FAKE + 8), ALIGN), (dict(gs=FAKE + 8), ALIGN), (dict(gg=FAKE + 2), ALIGN), (dict(uq=FAKE + 8), ALIGN),
    (dict(us=FAKE + 8), ALIGN), (dict(ug=FAKE + 2), ALIGN), (dict(dq=FAKE + 8), ALIGN), (dict(ds=FAKE + 8), ALIGN), (dict(dg=FAKE + 2), ALIGN),
    (dict(slot=FAKE + 2), ALIGN), (dict(weight=FAKE + 2), ALIGN), (dict(base=FAKE + 8), ALIGN), (dict(out=FAKE + 8), ALIGN), (dict(index=FAKE + 2), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 8), WORKSPACE), (dict(n=1000), WORKSPACE)])
def test_mlp_argument_errors(nv, change, status):
    assert mlp(nv, **change) == status


def test_mlp_accepts(nv):
    for change in (dict(), dict(base=None), dict(gq=None, gs=None, gg=None), dict(tokens=0, rows=0, x=None, out=None, index=None)):
        assert mlp(nv, **change) in PAST


def test_wrappers_refuse(nv):
    """What the wrappers check themselves; tensors of the CPU never reach the library."""
    c = nv.kv_cache(2, 2, 16, 64, device="cpu")
    assert c.q.shape == (2, 2, 2, 16, 32) and c.sf.shape == (2, 2, 2, 16, 4) and c.g.tolist() == [1.0, 1.0]
    assert nv.kv_cache(1, 1, 16, 64, 0.0, 5.5, device="cpu").g[0] == 1
    keys, values = c.keys(), c.values()
    assert keys.rows == 64 and keys.k == 64 and keys.q.data_ptr() == c.q.data_ptr() and keys.sf.shape == (64, 4)
    assert values.q.data_ptr() == c.q[1].data_ptr() and values.sf.data_ptr() == c.sf[1].data_ptr() and values.g.data_ptr() == c.g[1:].data_ptr()
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    table, place = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        nv.kv_append(c, x, x, table, place)
    with pytest.raises(ValueError, match="CUDA"):
        nv.kv_attention(x[:, None], c, table, place)
    r = nv.Routing(*(place,) * 5, None)
    w = nv.NVFP4Tensor(place, place, place, 1, 1, 0)
    with pytest.raises(ValueError, match="CUDA"):
        nv.expert_mlp(x[:, 0], r, w, w)


def test_wrappers_refuse_workspaces_that_are_not_contiguous(nv, monkeypatch):
    """A byte expanded to the size asked for: its elements are counted, but there is one."""
    monkeypatch.setattr(nv, "_one_device", lambda name, *t: t[0].device)
    monkeypatch.setattr(nv, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0)
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)  # noqa: E731
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    c = nv.kv_cache(2, 2, 16, 64, device="cpu")
    kv, table, place = z(3, 2, 64), z(3, 2, dtype=i32), z(3, dtype=i32)
    w = nv.NVFP4Tensor(z(2, 128, 64, dtype=u8), z(2 * 128 * 8, dtype=u8), z(2, dtype=f32), 128, 128, nv.NVFP4_SF_MMA)
    w.n = 128
    x, off, slots, weight = z(3, 128), z(3, dtype=i32), z(3, 1, dtype=i32), z(3, 1, dtype=f32)
    r = nv.Routing(slots, weight, off, place, slots, None)
    calls = [lambda ws: nv.kv_append(c, kv, kv, table, place, workspace=ws),
             lambda ws: nv.kv_attention(kv[:, None], c, table, place, workspace=ws),
             lambda ws: nv.expert_mlp(x, r, w, w, workspace=ws),
             lambda ws: nv.grouped_gemv(off, x, w.q, w.sf, w.g, 128, workspace=ws),
             lambda ws: nv.combine(x, slots, weight, workspace=ws),
             lambda ws: nv.combine_backward(x, x, slots, weight, off, workspace=ws),
             lambda ws: nv.route(z(3, 2, dtype=f32), 1, workspace=ws),
             lambda ws: nv.rmsnorm_backward(x, x, z(128), z(3, dtype=f32), workspace=ws)]
    a = nv.NVFP4Tensor(z(128, 64, dtype=u8), z(128 * 8, dtype=u8), z(1, dtype=f32), 128, 128, nv.NVFP4_SF_MMA)
    codes, e8 = z(128, 128, dtype=u8), z(128 * 4, dtype=u8)
    calls += [lambda ws: nv.gemm(a, a, workspace=ws, stream=0),
              lambda ws: nv.grouped_gemm(z(2, dtype=i32), a, a.q[None], a.sf, a.g, 128, workspace=ws, stream=0),
              lambda ws: nv.mx_gemm(codes, e8, codes, e8, workspace=ws, stream=0),
              lambda ws: nv.mx4_gemm(codes, e8, codes, e8, workspace=ws, stream=0),
              lambda ws: nv.gather_rows(a, z(5, dtype=i32), workspace=ws, stream=0)]
    for call in calls:
        for ws in (z(1, dtype=u8).expand(1 << 24), z(1 << 12, dtype=u8)[::2]):
            with pytest.raises(ValueError, match="contiguous workspace"):
                call(ws)
        with pytest.raises(nv.NVFP4Error, match="no sm_100|unsupported|CUDA"):  # (every check passed: no device)
            call(z(1 << 24, dtype=u8))
