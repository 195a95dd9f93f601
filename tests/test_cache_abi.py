"""The resident 8-bit cache's host side without a GPU: argument checks,
workspace plan and batch validation.  The device addresses below are never
dereferenced: a refused call enqueues nothing."""
import ctypes
import subprocess
import sys

import numpy as np
import pytest

import kv_cache_page_kvc_amd as kvc

FAKE = 1 << 40
CTX = ctypes.c_void_p(16)


def cache(H=4, D=128, T=16, P=64, **more):
    c = kvc.kvc_cache(kvc.KVC_ABI_VERSION, kvc.KVC_FP8_DYNAMIC, H, D, T, 0, P, H * T * D, H, FAKE, FAKE + (1 << 32),
                      FAKE + (1 << 33), FAKE + (1 << 34))
    for k, v in more.items():
        setattr(c, k, v)
    return c


def batch(n_seqs=3, n_rows=10, max_rows=6, max_len=100, columns=8, **more):
    b = kvc.kvc_batch(n_seqs, n_rows, max_rows, max_len, columns, FAKE + (1 << 35), FAKE + (1 << 36), FAKE + (1 << 37), None)
    for k, v in more.items():
        setattr(b, k, v)
    return b


def rows(heads=4, D=128, dtype=kvc.KVC_BF16, **more):
    r = kvc.kvc_rows(dtype, heads, heads * D, D, FAKE + (1 << 38))
    for k, v in more.items():
        setattr(r, k, v)
    return r


def options(q_heads=8, flags=1, window=0, scale=0.1):
    return kvc.kvc_attend(q_heads, flags, window, scale)


def R(x):
    return ctypes.byref(x) if x is not None else None


def write(c=None, b=None, k=None, v=None, ctx=None, fn="kvc_cache_write"):
    return getattr(kvc.lib(), fn)(ctx, R(c or cache()), R(b or batch()), R(k or rows()), R(v or rows()), None)


def attend(c=None, b=None, o=None, q=None, out=None, ws=None, ws_bytes=0, lse=None, ctx=None):
    return kvc.lib().kvc_cache_attend(ctx, R(c or cache()), R(b or batch()), R(o or options()), R(q or rows(8)),
                                      R(out or rows(8)), lse, ws, ws_bytes, None)


BAD_CACHES = [
    (dict(abi=1), kvc.KVC_E_ARG), (dict(reserved=1), kvc.KVC_E_ARG), (dict(codec=kvc.CODECS["FP8_DIRECT"]), kvc.KVC_E_UNSUPPORTED),
    (dict(codec=99), kvc.KVC_E_UNSUPPORTED), (dict(head_dim=96), kvc.KVC_E_UNSUPPORTED), (dict(head_dim=512), kvc.KVC_E_UNSUPPORTED),
    (dict(tokens_per_page=8), kvc.KVC_E_UNSUPPORTED), (dict(tokens_per_page=48), kvc.KVC_E_UNSUPPORTED),
    (dict(tokens_per_page=512, stride_page=1 << 30), kvc.KVC_E_UNSUPPORTED), (dict(kv_heads=0), kvc.KVC_E_ARG),
    (dict(num_pages=0), kvc.KVC_E_ARG), (dict(num_pages=1 << 31), kvc.KVC_E_ARG), (dict(stride_page=4 * 16 * 128 - 16), kvc.KVC_E_ARG),
    (dict(stride_page=4 * 16 * 128 + 8), kvc.KVC_E_ARG), (dict(stride_page=1 << 32), kvc.KVC_E_UNSUPPORTED), (dict(stride_scale=1 << 32), kvc.KVC_E_UNSUPPORTED), (dict(stride_scale=3), kvc.KVC_E_ARG),
    (dict(k_codes=None), kvc.KVC_E_ARG), (dict(v_codes=FAKE + 8), kvc.KVC_E_ARG), (dict(k_scales=FAKE + 2), kvc.KVC_E_ARG),
    (dict(v_scales=None), kvc.KVC_E_ARG),
]
BAD_BATCHES = [
    dict(n_seqs=(1 << 20) + 1), dict(n_rows=(1 << 30) + 1), dict(max_len=8 * 16 + 1), dict(max_len=(1 << 30) + 1, stride_table=1 << 27),
    dict(stride_table=-1), dict(cu_rows=None), dict(lengths=None), dict(block_table=None), dict(cu_rows=FAKE + 2), dict(seq_flags=FAKE + 1),
]
BAD_ROWS = [
    (dict(dtype=3), kvc.KVC_E_UNSUPPORTED), (dict(heads=5), kvc.KVC_E_ARG), (dict(stride_row=0), kvc.KVC_E_ARG),
    (dict(stride_head=-128), kvc.KVC_E_ARG), (dict(stride_row=4 * 128 + 4), kvc.KVC_E_ARG), (dict(stride_head=132), kvc.KVC_E_ARG),
    (dict(stride_row=1 << 62), kvc.KVC_E_ARG), (dict(data=None), kvc.KVC_E_ARG), (dict(data=FAKE + 8), kvc.KVC_E_ARG),
]


@pytest.mark.parametrize("fn", ["kvc_cache_write", "kvc_cache_read"])
def test_rows_calls_refuse_bad_arguments(fn):
    for bad, st in BAD_CACHES:
        assert write(c=cache(**bad), fn=fn) == st, bad
    for bad in BAD_BATCHES:
        assert write(b=batch(**bad), fn=fn) == kvc.KVC_E_ARG, bad
    for bad, st in BAD_ROWS:
        assert write(k=rows(**bad), fn=fn) == st, bad
        assert write(v=rows(**bad), fn=fn) == st, bad
    assert write(k=rows(dtype=kvc.KVC_FP16), fn=fn) == kvc.KVC_E_ARG                  # K and V of one type
    assert write(fn=fn) == kvc.KVC_E_ARG                                              # all well but no context
    L = getattr(kvc.lib(), fn)
    ok = [R(cache()), R(batch()), R(rows()), R(rows())]
    for i in range(4):
        assert L(CTX, *[None if i == j else x for j, x in enumerate(ok)], None) == kvc.KVC_E_ARG
    # nothing to do: no device is touched
    assert write(b=batch(n_seqs=0), ctx=CTX, fn=fn) == kvc.KVC_OK
    assert write(b=batch(n_rows=0), k=rows(data=None), v=rows(data=None), ctx=CTX, fn=fn) == kvc.KVC_OK


def test_launches_that_are_too_large_are_refused():
    huge = dict(n_seqs=1, n_rows=1 << 30, max_rows=1 << 30, max_len=1 << 30, stride_table=1 << 26)
    for fn in ("kvc_cache_write", "kvc_cache_read"):
        assert write(b=batch(**huge), fn=fn, ctx=CTX) == kvc.KVC_E_ARG
    assert attend(b=batch(n_seqs=1 << 20, n_rows=1 << 29, max_rows=1 << 20, max_len=1 << 12, stride_table=1 << 8),
                  q=rows(4), out=rows(4), o=options(q_heads=4), ctx=CTX) == kvc.KVC_E_ARG


def test_outputs_must_not_overlap():
    half = dict(stride_row=2 * 128)                        # rows of 4 heads x 128 at half their size
    assert write(k=rows(**half), fn="kvc_cache_read") == kvc.KVC_E_ARG
    assert attend(out=rows(8, stride_row=4 * 128)) == kvc.KVC_E_ARG
    assert attend(out=rows(8, stride_head=64, stride_row=4096)) == kvc.KVC_E_ARG
    by_head = dict(stride_row=128, stride_head=10 * 128)   # [heads][rows][D] does not: only the context is missing
    assert write(k=rows(**by_head), v=rows(**by_head), b=batch(n_seqs=0), ctx=CTX, fn="kvc_cache_read") == kvc.KVC_OK


def test_attend_refuses_bad_arguments():
    for bad, st in BAD_CACHES:
        assert attend(c=cache(**bad)) == st, bad
    for bad in BAD_BATCHES:
        assert attend(b=batch(**bad)) == kvc.KVC_E_ARG, bad
    for bad, st in BAD_ROWS:
        bad = {k: (v + 4 * 128 if k == "stride_row" and v == 4 * 128 + 4 else v) for k, v in bad.items()}
        assert attend(q=rows(8, **{k: v for k, v in bad.items() if k != "heads"}) if "heads" not in bad else rows(5)) == st, bad
        assert attend(out=rows(8, **{k: v for k, v in bad.items() if k != "heads"}) if "heads" not in bad else rows(5)) == st, bad
    for o in (options(q_heads=0), options(q_heads=6), options(flags=2), options(scale=0.0), options(scale=-1.0),
              options(scale=float("nan")), options(scale=float("inf"))):
        assert attend(o=o) == kvc.KVC_E_ARG, (o.q_heads, o.flags, o.scale)
    assert attend(out=rows(8, dtype=kvc.KVC_FP16)) == kvc.KVC_E_ARG
    assert attend(lse=ctypes.c_void_p(FAKE + 2)) == kvc.KVC_E_ARG
    assert attend() == kvc.KVC_E_ARG                                                  # no context
    assert attend(b=batch(n_seqs=0), ctx=CTX) == kvc.KVC_OK
    # more rows x heads than the kernels count in 32 bits
    big = batch(n_rows=1 << 30, max_rows=1 << 30)
    assert attend(b=big, o=options(q_heads=8)) == kvc.KVC_E_ARG


def test_attend_workspace():
    n = ctypes.c_size_t(7)
    L = kvc.lib()
    c, o = cache(P=1 << 20), options()
    # short contexts are not split
    assert L.kvc_plan_attend(R(c), R(batch()), R(o), ctypes.byref(n)) == kvc.KVC_OK and n.value == 0
    long = batch(n_seqs=2, n_rows=2, max_rows=1, max_len=100000, columns=8192)
    assert L.kvc_plan_attend(R(c), R(long), R(o), ctypes.byref(n)) == kvc.KVC_OK
    per_split = 2 * 8 * (128 + 2) * 4
    assert n.value > per_split and n.value % per_split == 0
    assert attend(c=c, b=long, ws=ctypes.c_void_p(FAKE), ws_bytes=n.value - 1, ctx=CTX) == kvc.KVC_E_CAPACITY
    assert attend(c=c, b=long, ws=None, ws_bytes=n.value, ctx=CTX) == kvc.KVC_E_ARG
    assert attend(c=c, b=long, ws=ctypes.c_void_p(FAKE + 4), ws_bytes=n.value, ctx=CTX) == kvc.KVC_E_ARG
    assert L.kvc_plan_attend(R(cache(head_dim=96)), R(long), R(o), ctypes.byref(n)) == kvc.KVC_E_UNSUPPORTED
    assert L.kvc_plan_attend(R(c), R(long), R(o), None) == kvc.KVC_OK


def test_validate_batch():
    c, b = cache(), batch(max_len=128)
    table = np.arange(24, dtype=np.int32).reshape(3, 8)
    cu, ln = np.array([0, 1, 6, 10], np.int32), np.array([1, 40, 128], np.int32)

    def check(table=table, cu=cu, ln=ln, writes=1, b=b):
        t, x, y = (np.ascontiguousarray(a, np.int32) for a in (table, cu, ln))
        return kvc.lib().kvc_validate_batch(R(c), R(b), t.ctypes.data, x.ctypes.data, y.ctypes.data, writes)

    assert check() == kvc.KVC_OK
    assert check(cu=[0, 7, 8, 10]) == kvc.KVC_E_ARG and check(cu=[0, 3, 2, 6]) == kvc.KVC_E_ARG
    assert check(cu=[-1, 1, 6, 10]) == kvc.KVC_E_ARG and check(cu=[0, 1, 6, 11]) == kvc.KVC_E_ARG
    assert check(ln=[1, 40, 129]) == kvc.KVC_E_ARG and check(ln=[-1, 40, 128]) == kvc.KVC_E_ARG
    t = table.copy()
    t[1, 2] = 64
    assert check(t) == kvc.KVC_E_PAGE_RANGE                # positions 32 .. 39 lie there
    t[1, 2], t[1, 3] = 10, -1                              # column 3 is behind the sequence
    assert check(t) == kvc.KVC_OK
    t[2, 7] = 10                                           # both sequences write page 10
    assert check(t) == kvc.KVC_E_DUP_DST and check(t, writes=0) == kvc.KVC_OK
    t[2, 7], t[2, 0] = 23, 10                              # a shared page that is only read
    assert check(t) == kvc.KVC_OK
    assert check(b=batch(max_len=129)) == kvc.KVC_E_ARG    # more than eight pages
    for i in range(3):
        a = [x.ctypes.data for x in (table, cu, ln)]
        a[i] = None
        assert kvc.lib().kvc_validate_batch(R(c), R(b), *a, 1) == kvc.KVC_E_ARG


def test_binding_checks():
    torch = pytest.importorskip("torch")
    kv = kvc.Cache.empty(4, 2, 64, 16, "INT8", device="cpu")
    assert kv.c.stride_page == 2 * 16 * 64 and kv.c.codec == kvc.KVC_INT8
    k, v, ks, vs = kv.tensors
    for bad in ((k.float(), v, ks, vs), (k, k, ks, vs), (k, v, ks.double(), vs), (k, v, ks[:2], vs),
                (k.view(torch.float8_e4m3fn), v, ks, vs), (k[:, :, :, ::1].transpose(0, 1).contiguous().transpose(0, 1), v, ks, vs)):
        with pytest.raises(ValueError):
            kvc.Cache(*bad)
    i32 = dict(dtype=torch.int32)
    table, cu, ln = torch.zeros((2, 3), **i32), torch.zeros(3, **i32), torch.zeros(2, **i32)
    b = kvc.Batch(table, cu, ln, 5, 5, 48)
    assert b.c.stride_table == 3
    for bad in ((table.long(), cu, ln), (table, cu[:2], ln), (table[:1], cu, ln), (table.t().contiguous().t(), cu, ln)):
        with pytest.raises(ValueError):
            kvc.Batch(*bad, 5, 5, 48)
    with pytest.raises(ValueError):
        kvc.Rows(torch.zeros(5, 2, 64, dtype=torch.bfloat16).transpose(1, 2))
    with pytest.raises(ValueError):
        kvc.Rows(torch.zeros(5, 2, 64))
    r = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                        # fewer rows than the batch's
        kvc.kvc_cache_write(None, kv, b, r, r)
    # a strided table: only its own columns may be read
    wide = torch.zeros((2, 9), **i32)[:, :3]
    with pytest.raises(kvc.KvcError):
        kvc.kvc_cache_read(None, kv, kvc.Batch(wide, cu, ln, 5, 5, 49), r, r)
    assert kvc.kvc_validate_batch(kv, kvc.Batch(wide, cu, ln, 5, 5, 48), wide, cu, [0, 0], True) == kvc.KVC_OK


def test_under_sanitizers(tmp_path_factory):
    """The checks above against the host half built with the sanitizers."""
    san = pytest.importorskip("tests.test_sanitizers")
    rt, oracle, host, _ = san.builds.__wrapped__(tmp_path_factory) if hasattr(san.builds, "__wrapped__") else \
        san.builds.__pytest_wrapped__.obj(tmp_path_factory)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", __file__, "-k",
                        "not sanitizers"], capture_output=True, text=True, env=san._env(rt, oracle, host),
                       cwd=san.ROOT, timeout=900)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0 and " passed" in r.stdout, out[-4000:]
