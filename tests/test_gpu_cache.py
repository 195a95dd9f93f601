"""The resident 8-bit cache on the GPU against its plain CPU reference
(tests/cache_reference.py): writes bit for bit, over the whole pool, reads bit
for bit, attention against 64 bits within the bound that its roundings give.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():      # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import kv_cache_page_kvc_amd as kvc                      # noqa: E402
from tests import cache_reference as ref                 # noqa: E402

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def ctx():
    c = kvc.kvc_create(0, 0)
    yield c
    torch.cuda.synchronize()
    kvc.kvc_destroy(c)


class World:
    """A cache on the GPU and its host double, with sequences in shuffled pages."""

    def __init__(self, codec, heads, dim, tokens, lengths, dtype="bf16", seed=0, spare=3):
        self.codec, self.H, self.D, self.T, self.dt = codec, heads, dim, tokens, DTYPES[dtype]
        self.rng = np.random.default_rng(seed)
        need = [-(-max(n, 0) // tokens) for n in lengths]
        pages = sum(need) + spare
        self.host = ref.Pool(pages, heads, tokens, dim, codec, seed)
        ids = self.rng.permutation(pages)
        columns = max(need + [1])
        # entries behind a sequence's pages are never followed
        self.table = np.full((len(lengths), columns), 0x7FFFFFFF, np.int64)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.dev = self.host.tensors("cuda")
        self.cache = kvc.Cache(*self.dev)

    def batch(self, rows, lengths, n_rows=None, max_rows=None, max_len=None, flags=None):
        cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
        i32 = [torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda") for x in (self.table, cu, lengths)]
        b = kvc.Batch(*i32, n_rows if n_rows is not None else int(cu[-1]),
                      max_rows if max_rows is not None else max(list(rows) + [0]),
                      max_len if max_len is not None else self.table.shape[1] * self.T, flags)
        return b, cu

    def values(self, n, heads=None, scale=1.0):
        x = self.rng.standard_normal((n, heads or self.H, self.D)) * scale
        x *= np.exp(self.rng.standard_normal((1, heads or self.H, self.D)))
        return torch.from_numpy(x.astype(np.float32)).to(self.dt)

    def check_pool(self, what=""):
        torch.cuda.synchronize()
        k, v, ks, vs = self.dev
        for name, got, want in (("k", k, self.host.k), ("v", v, self.host.v.transpose(0, 1, 3, 2))):
            got = got.view(torch.uint8).cpu().numpy()
            bad = np.argwhere(got != want)
            assert not len(bad), f"{what} {name}: {len(bad)} codes differ, first at {bad[0]}: " \
                                 f"{got[tuple(bad[0])]} for {want[tuple(bad[0])]}"
        for name, got, want in (("k", ks, self.host.ks), ("v", vs, self.host.vs)):
            got = got.cpu().numpy()
            assert np.array_equal(got.view(np.uint32), want.view(np.uint32)), f"{what} {name} scales differ"

    def write(self, ctx, rows, lengths, k=None, v=None, stream=0, **bounds):
        b, cu = self.batch(rows, lengths, **bounds)
        n = int(cu[-1])
        k = self.values(n) if k is None else k
        v = self.values(n) if v is None else v
        kvc.kvc_cache_write(ctx, self.cache, b, k.cuda(), v.cuda(), stream)
        odd = self.host.write(self.table, cu, lengths, k.float().numpy(), v.float().numpy())
        return b, cu, odd

    def widen(self, columns):
        """A wider block table, so that batches promise longer contexts than there are: other kernels and splits."""
        more = np.full((self.table.shape[0], max(columns - self.table.shape[1], 0)), 0x7FFFFFFF, np.int64)
        self.table = np.concatenate([self.table, more], 1)

    def fill(self, ctx, lengths):
        self.write(ctx, lengths, lengths)
        self.check_pool("fill")

    def attend(self, ctx, rows, lengths, group, causal=True, window=0, scale=None, q=None, lse=True, hidden=(),
               **bounds):
        b, cu = self.batch(rows, lengths, **bounds)
        n, Hq = int(cu[-1]), self.H * group
        q = self.values(n, Hq) if q is None else q
        out = torch.full((n, Hq, self.D), 7.0, dtype=self.dt, device="cuda")
        z = torch.full((n, Hq), 7.0, device="cuda") if lse else None
        o = kvc.Attend(Hq, causal, window, scale)
        need = kvc.kvc_plan_attend(self.cache, b, o)
        ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")     # NaN everywhere
        kvc.kvc_cache_attend(ctx, self.cache, b, o, q.cuda(), out, z, ws)
        torch.cuda.synchronize()
        want, want_z, off, off_z = ref.attend(self.host, self.table, cu, lengths, q.float().numpy(),
                                              scale or self.D ** -0.5, causal, window, hidden)
        self.compare(out, z, want, want_z, off, off_z)
        return out, z, need

    def compare(self, out, z, want, want_z, off, off_z):
        got = out.double().cpu().numpy()
        allowed = ref.tolerance(want, off, self.dt)
        err = np.abs(got - want)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and not np.isinf(got).any()
        worst = np.nanmax(err / allowed) if err.size else 0.0
        assert worst <= 1.0, f"off by {worst:.2f} of what the roundings allow at {np.unravel_index(np.nanargmax(err / allowed), err.shape)}"
        if z is not None:
            g = z.double().cpu().numpy()
            assert np.array_equal(g == -np.inf, want_z == -np.inf)
            fin = np.isfinite(want_z)
            far = np.abs(g[fin] - want_z[fin])
            assert (far <= off_z[fin]).all(), far.max()


# ------------------------------------------------------------------ write
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("codec", ["FP8_DYNAMIC", "INT8"])
@pytest.mark.parametrize("D,T,H", [(32, 16, 3), (64, 32, 2), (128, 16, 8), (128, 64, 1), (256, 16, 2), (256, 128, 1),
                                   (64, 256, 2)])
def test_write_prompts_then_append(ctx, codec, dtype, D, T, H):
    print(f"[case] write {codec} {dtype} D={D} T={T} H={H}", flush=True)
    final = [1, T - 1, T, T + 1, 2 * T + 7, 3, 40]
    w = World(codec, H, D, T, [n + 9 for n in final], dtype, seed=D + T)
    w.write(ctx, final, final)
    w.check_pool("prompt")
    lengths = list(final)
    for step, rows in enumerate(([1] * 7, [1] * 7, [5, 0, 3, 1, 2, 0, 7])):
        lengths = [a + b for a, b in zip(lengths, rows)]
        # the second step's values outgrow the scales: earlier codes are quantised anew
        k, v = (w.values(sum(rows), scale=(1.0, 9.0, 0.01)[step]) for _ in range(2))
        w.write(ctx, rows, lengths, k, v)
        w.check_pool(f"append {step}")


@pytest.mark.parametrize("codec", ["FP8_DYNAMIC", "INT8"])
def test_write_specials(ctx, codec):
    """NaN, infinities, zeros, denormals and the largest values, fresh and appended; sequences are flagged."""
    for dtype in ("bf16", "fp16"):
        w = World(codec, 2, 64, 16, [40] * 5, dtype, seed=5)
        top = torch.finfo(w.dt).max
        flags = torch.zeros(5, dtype=torch.int32, device="cuda")
        for start, n in ((0, 20), (20, 1), (21, 16)):
            rows = [n] * 5
            k, v = w.values(5 * n), w.values(5 * n)
            for x in (k, v):
                y = x.view(5, n, 2, 64)
                y[0, :, 0] = 0.0                           # an empty block
                y[1, n // 2, 1, 3] = float("nan")
                y[1, n // 2, 1, 5] = float("-inf")
                y[2, n - 1, 0, 63] = float("inf")
                y[2, :, 1] = float("nan")                  # nothing finite
                y[3, 0, 0, 0] = top
                y[3, 0, 0, 1] = -top
                y[4, :, 0] = torch.finfo(w.dt).smallest_normal / 4
            _, _, odd = w.write(ctx, rows, [start + n] * 5, k, v, flags=flags)
            w.check_pool(f"{dtype} {start}")
            assert odd == {1, 2}
            assert flags.tolist() == [0, 4, 4, 0, 0]


def test_write_unwritten_page_start(ctx):
    """Appending to a page that nothing was written to (its scale is 0, NaN, infinite or negative) keeps no old code."""
    w = World("INT8", 4, 32, 16, [48] * 12, seed=3)
    w.write(ctx, [3] * 12, [8] * 12)
    w.check_pool()


def test_write_strided_rows_and_left_rows(ctx):
    """K and V as slices of a fused projection, heads-first rows, and rows behind the last sequence."""
    w = World("FP8_DYNAMIC", 4, 64, 16, [50, 30], "bf16", seed=9)
    rows, n = [50, 30], 80
    fused = torch.randn(n + 5, 16, 64).to(torch.bfloat16)
    b, cu = w.batch(rows, rows, n_rows=n + 5)
    dev = fused.cuda()
    kvc.kvc_cache_write(ctx, w.cache, b, dev[:, 8:12], dev[:, 12:16])
    w.host.write(w.table, cu, rows, fused[:, 8:12].float().numpy(), fused[:, 12:].float().numpy())
    w.check_pool("fused")
    heads = torch.randn(4, n, 64).to(torch.bfloat16)
    b, cu = w.batch(rows, rows)
    kvc.kvc_cache_write(ctx, w.cache, b, heads.cuda().transpose(0, 1), heads.cuda().transpose(0, 1))
    h = heads.transpose(0, 1).float().numpy()
    w.host.write(w.table, cu, rows, h, h)
    w.check_pool("heads first")


def test_write_strided_pool(ctx):
    """Pages of several layers interleaved: page strides beyond a page's own size."""
    w = World("INT8", 2, 64, 32, [70, 33], seed=4)
    P = w.host.k.shape[0]
    k, v, ks, vs = w.dev
    big = [torch.zeros((P, 3) + t.shape[1:], dtype=t.dtype, device="cuda") for t in (k, v, ks, vs)]
    for b_, t in zip(big, w.dev):
        b_[:, 1] = t
    w.dev = tuple(b_[:, 1] for b_ in big)
    w.cache = kvc.Cache(*w.dev)
    w.write(ctx, [70, 33], [70, 33])
    w.check_pool()
    assert not any(bool(b_[:, i].any()) for b_ in big for i in (0, 2))


@pytest.mark.parametrize("n_seqs", [1, 70, 5000])
def test_write_many_ragged_sequences(ctx, n_seqs):
    """Units found by search: one long sequence among short ones, empty ones and ones without rows."""
    rng = np.random.default_rng(n_seqs)
    rows = rng.integers(0, 4, n_seqs)
    rows[n_seqs // 2] = 300
    past = np.where(rng.random(n_seqs) < 0.5, 0, rng.integers(0, 20, n_seqs))
    lengths = (rows + past).tolist()
    w = World("INT8", 1, 32, 16, [max(n, 1) for n in lengths], seed=n_seqs)
    w.write(ctx, past.tolist(), past.tolist())
    w.check_pool("past")
    w.write(ctx, rows.tolist(), lengths, n_rows=int(rows.sum()))
    w.check_pool("rows")


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("codec", ["FP8_DYNAMIC", "INT8"])
@pytest.mark.parametrize("D,T,H", [(32, 32, 3), (64, 16, 2), (128, 16, 8), (256, 64, 2), (128, 256, 1)])
def test_read(ctx, codec, dtype, D, T, H):
    print(f"[case] read {codec} {dtype} D={D} T={T} H={H}", flush=True)
    lengths = [1, T, T + 5, 100, 2 * T + 1, 0]
    w = World(codec, H, D, T, lengths, dtype, seed=1)
    w.fill(ctx, lengths)
    for rows in (lengths, [1, 2, T, 37, T + 1, 0], [1, 0, 0, 100, 0, 0], [4, T + 3, 2, 1, 0, 2]):
        # the last list asks for more rows than positions: those are zero
        b, cu = w.batch(rows, lengths, n_rows=sum(rows) + 3)
        k, v = (torch.full((sum(rows) + 3, H, D), 7.0, dtype=w.dt, device="cuda") for _ in range(2))
        kvc.kvc_cache_read(ctx, w.cache, b, k, v)
        torch.cuda.synchronize()
        for got, want in zip((k, v), w.host.read(w.table, cu, lengths, sum(rows), w.dt)):
            assert torch.equal(got[:-3].cpu().view(torch.int16), want.view(torch.int16))
            assert bool((got[-3:] == 7.0).all())


def test_read_strided_destination(ctx):
    """Rows into every second head of a wider tensor; the rest stays."""
    w = World("FP8_DYNAMIC", 2, 64, 16, [21, 40], "fp16", seed=8)
    w.fill(ctx, [21, 40])
    b, cu = w.batch([21, 40], [21, 40])
    wide = torch.full((61, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    kvc.kvc_cache_read(ctx, w.cache, b, wide[:, 0:4:2], wide[:, 5:8:2])
    want = w.host.read(w.table, cu, [21, 40], 61, w.dt)
    assert torch.equal(wide[:, 0:4:2].cpu(), want[0]) and torch.equal(wide[:, 5:8:2].cpu(), want[1])
    assert bool((wide[:, [1, 3, 4, 6]] == 7.0).all())


# ------------------------------------------------------------------ attend
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("codec", ["FP8_DYNAMIC", "INT8"])
@pytest.mark.parametrize("D,T,H,G", [(32, 16, 2, 5), (64, 32, 3, 1), (128, 16, 2, 4), (128, 64, 1, 16), (256, 16, 1, 7),
                                     (256, 256, 2, 2)])
def test_attend_single_tokens(ctx, codec, dtype, D, T, H, G):
    print(f"[case] attend one {codec} {dtype} D={D} T={T} H={H} G={G}", flush=True)
    lengths = [1, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 700]
    w = World(codec, H, D, T, lengths, dtype, seed=2)
    w.fill(ctx, lengths)
    w.attend(ctx, [1] * 12, lengths, G)
    w.attend(ctx, [1] * 12, lengths, G, causal=False, lse=False)
    w.attend(ctx, [1] * 12, lengths, G, window=33)


@pytest.mark.parametrize("codec", ["FP8_DYNAMIC", "INT8"])
@pytest.mark.parametrize("D,T,H,G", [(32, 64, 1, 3), (64, 16, 2, 4), (128, 32, 2, 2), (128, 16, 1, 1), (256, 16, 1, 5)])
def test_attend_prompts_and_chunks(ctx, codec, D, T, H, G):
    print(f"[case] attend rows {codec} D={D} T={T} H={H} G={G}", flush=True)
    lengths = [200, 65, 129, 16, 300, 7]
    w = World(codec, H, D, T, lengths, "bf16", seed=6)
    w.fill(ctx, lengths)
    for columns in (0, 2200 // T):                                        # few rows a tile, then many
        w.widen(columns)
        w.attend(ctx, lengths, lengths, G)                                # whole prompts
        w.attend(ctx, [33, 1, 128, 3, 77, 0], lengths, G)                 # chunks behind a past
        w.attend(ctx, [5, 5, 2, 5, 5, 5], lengths, G, window=20)          # drafts with a window
        w.attend(ctx, lengths, lengths, G, window=70)
        w.attend(ctx, [40, 65, 3, 16, 9, 7], lengths, G, causal=False)
        w.attend(ctx, [40, 65, 3, 16, 9, 7], lengths, G, causal=False, window=11)


@pytest.mark.parametrize("codec,D,H,G,dtype", [("INT8", 128, 2, 4, "fp16"), ("FP8_DYNAMIC", 64, 1, 8, "bf16"),
                                               ("FP8_DYNAMIC", 256, 1, 3, "fp16"), ("INT8", 32, 3, 5, "bf16")])
def test_attend_many_rows(ctx, codec, D, H, G, dtype):
    """Several tiles of many rows, several splits, ragged: ends that fall inside tiles, waves without rows."""
    print(f"[case] attend many {codec} D={D} H={H} G={G}", flush=True)
    lengths = [2600, 130, 700, 1, 0]
    w = World(codec, H, D, 32, lengths, dtype, seed=21)
    w.fill(ctx, lengths)
    w.attend(ctx, [300, 130, 257, 1, 0], lengths, G)
    w.attend(ctx, [97, 64, 40, 1, 0], lengths, G, window=600)
    w.widen(400)                                           # 12,800 positions promised: a split sees nothing
    w.attend(ctx, [300, 130, 257, 1, 0], lengths, G)


@pytest.mark.parametrize("codec,D,H,G,rows", [("INT8", 128, 1, 8, 60), ("FP8_DYNAMIC", 64, 2, 4, 90),
                                              ("INT8", 256, 4, 5, 100)])
def test_attend_many_rows_many_splits(ctx, codec, D, H, G, rows):
    """Many rows behind a long context: up to 20 splits, some of which the shorter sequence does not have."""
    lengths = [20000, 2500]
    w = World(codec, H, D, 64, lengths, "bf16", seed=41)
    w.fill(ctx, lengths)
    w.attend(ctx, [rows, 33], lengths, G)
    w.attend(ctx, [rows, 33], lengths, G, window=3000)


@pytest.mark.parametrize("rows,length", [(380, 380), (400, 400), (480, 700), (720, 720)])
def test_attend_one_prompt_of_some_rounds(ctx, rows, length):
    """One sequence of 8 to 15 tiles a head: with 64 heads 2 to 4 rounds of workgroups, whose order is not the tiles'."""
    w = World("FP8_DYNAMIC", 64, 128, 16, [length], "bf16", seed=31)
    w.fill(ctx, [length])
    w.attend(ctx, [rows], [length], 8)


def test_attend_long_context_splits(ctx):
    """One sequence of 40,000 positions among short ones, split and joined."""
    for codec, lengths, G in (("INT8", [40000], 4), ("FP8_DYNAMIC", [9000, 3, 4097, 1], 8)):
        w = World(codec, 1, 128, 16, lengths, "fp16", seed=7)
        w.fill(ctx, lengths)
        _, _, need = w.attend(ctx, [1] * len(lengths), lengths, G)
        assert need > 0
        w.attend(ctx, [min(3, n) for n in lengths], lengths, G, window=5000)
        # bounds far above the lengths change the cut, not the result
        w.table = np.concatenate([w.table, np.zeros((len(lengths), 5000), np.int64)], 1)
        w.attend(ctx, [1] * len(lengths), lengths, G)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attend_rows_that_see_nothing(ctx, dtype):
    """Empty sequences, rows before position 0, and rows behind the last sequence."""
    lengths = [0, 3, 100, 5]
    w = World("INT8", 2, 64, 16, lengths, dtype, seed=11)
    w.fill(ctx, lengths)
    for rows in ([2, 7, 1, 5], [2, 7, 40, 9], [300, 0, 0, 5], [40, 7, 40, 9]):
        for causal in (True, False):
            w.widen(200 if rows[0] == 40 else 0)
            out, z, _ = w.attend(ctx, rows, lengths, 3, causal=causal)
            assert bool((out[:2] == 0).all()) and bool((z[:2] == -float("inf")).all())
            if causal and rows[1] == 7:
                assert bool((out[2:6] == 0).all())
    b, cu = w.batch([1, 1, 1, 1], lengths, n_rows=9, max_rows=9)
    out = torch.full((9, 6, 64), 7.0, dtype=w.dt, device="cuda")
    z = torch.full((9, 6), 7.0, device="cuda")
    kvc.kvc_cache_attend(ctx, w.cache, b, kvc.Attend(6), w.values(9, 6).cuda(), out, z,
                         torch.zeros(kvc.kvc_plan_attend(w.cache, b, kvc.Attend(6)) + 16, dtype=torch.uint8, device="cuda"))
    assert bool((out[4:] == 7.0).all()) and bool((z[4:] == 7.0).all()) and not bool((out[1:4] == 7.0).any())


def test_pages_before_the_window_may_be_gone(ctx):
    """Table entries that no row looks at any more are neither followed nor reported."""
    w = World("INT8", 1, 64, 16, [300, 90], seed=24)
    w.fill(ctx, [300, 90])
    real = w.table.copy()
    for rows, columns in (([1, 1], 0), ([20, 33], 200)):
        w.table = real.copy()
        w.widen(columns)
        flags = torch.zeros(2, dtype=torch.int32, device="cuda")
        for b in range(2):
            first = [300, 90][b] - rows[b] - 30 + 1        # the first position that a row sees
            w.table[b, :first // 16] = -1
        gone = w.table
        b, cu = w.batch(rows, [300, 90], flags=flags)
        q = w.values(sum(rows), 2)
        out, z = torch.zeros((sum(rows), 2, 64), dtype=w.dt, device="cuda"), torch.zeros((sum(rows), 2), device="cuda")
        o = kvc.Attend(2, window=30)
        ws = torch.zeros(kvc.kvc_plan_attend(w.cache, b, o) + 16, dtype=torch.uint8, device="cuda")
        kvc.kvc_cache_attend(ctx, w.cache, b, o, q.cuda(), out, z, ws)
        assert flags.tolist() == [0, 0] and gone[0, 0] == -1
        w.compare(out, z, *ref.attend(w.host, real, cu, [300, 90], q.float().numpy(), 64 ** -0.5, True, 30))


def test_nothing_cached(ctx):
    """max_len 0 and a block table without columns: rows come back empty, writes store nothing."""
    w = World("FP8_DYNAMIC", 2, 32, 16, [0, 0], "fp16", seed=25)
    i32 = dict(dtype=torch.int32, device="cuda")
    b = kvc.Batch(torch.zeros((2, 0), **i32), torch.tensor([0, 3, 5], **i32), torch.zeros(2, **i32), 5, 3, 0)
    k, v = (torch.full((5, 2, 32), 7.0, dtype=w.dt, device="cuda") for _ in range(2))
    kvc.kvc_cache_write(ctx, w.cache, b, k, v)
    w.check_pool()
    kvc.kvc_cache_read(ctx, w.cache, b, k, v)
    assert not bool(k.any()) and not bool(v.any())
    for heads in (2, 64):
        q = w.values(5, heads)
        out, z = torch.full((5, heads, 32), 7.0, dtype=w.dt, device="cuda"), torch.zeros((5, heads), device="cuda")
        kvc.kvc_cache_attend(ctx, w.cache, b, kvc.Attend(heads), q.cuda(), out, z)
        assert not bool(out.any()) and bool((z == -float("inf")).all())


def test_attend_ignores_what_was_not_written(ctx):
    """The last page's unwritten tokens hold NaN codes, and pages behind the sequence NaN scales."""
    w = World("FP8_DYNAMIC", 1, 64, 32, [70], seed=12)
    w.fill(ctx, [70])
    page = int(w.table[0, 2])
    w.dev[0].view(torch.uint8)[page, :, 6:] = 0x7F
    w.dev[1].view(torch.uint8)[page, :, :, 6:] = 0xFF
    w.attend(ctx, [1], [70], 2)
    w.attend(ctx, [70], [70], 2)
    w.attend(ctx, [3], [64], 2)                            # a shorter length hides the third page
    w.widen(100)
    w.attend(ctx, [70], [70], 2)
    w.attend(ctx, [64], [64], 2)


@pytest.mark.parametrize("columns", [0, 200], ids=["few", "many"])
def test_attend_query_specials(ctx, columns):
    """A row of zeros, tiny and huge rows, and NaN / infinite rows, which are NaN by themselves."""
    lengths = [50]
    for dtype in ("bf16", "fp16"):
        w = World("INT8", 1, 128, 16, lengths, dtype, seed=13)
        w.fill(ctx, lengths)
        w.widen(columns)
        q = w.values(6 if not columns else 40, 2)
        q[0] = 0.0
        q[1] = q[1] * 1e-6
        q[1, 0, 5] = torch.finfo(w.dt).smallest_normal / 8
        q[3, 1, 7] = float("nan")
        q[4, 0, 100] = float("inf")
        n = q.shape[0]
        b, cu = w.batch([n], lengths)
        out = torch.zeros((n, 2, 128), dtype=w.dt, device="cuda")
        z = torch.zeros((n, 2), device="cuda")
        o = kvc.Attend(2)
        ws = torch.zeros(kvc.kvc_plan_attend(w.cache, b, o) + 16, dtype=torch.uint8, device="cuda")
        kvc.kvc_cache_attend(ctx, w.cache, b, o, q.cuda(), out, z, ws)
        bad = torch.zeros(n, 2, dtype=torch.bool)
        bad[3, 1] = bad[4, 0] = True
        assert torch.equal(out.cpu().isnan(), bad[..., None].expand(-1, -1, 128))
        assert torch.equal(z.cpu().isnan(), bad)
        clean = torch.where(bad[..., None], torch.zeros((), dtype=w.dt), q)
        want = ref.attend(w.host, w.table, cu, lengths, clean.float().numpy(), 128 ** -0.5, True, 0)
        keep = ~bad.numpy()
        w.compare(out[~bad.cuda()], z[~bad.cuda()], *(x[keep] for x in want))


def test_shared_prefix_and_repeated_pages(ctx):
    """Two sequences read the same pages, one of them a page twice; each writes its own last page."""
    w = World("FP8_DYNAMIC", 2, 64, 16, [48, 48], seed=22)
    w.fill(ctx, [48, 48])
    w.table[1, :2] = w.table[0, 0]
    w.attend(ctx, [1, 1], [48, 48], 4)
    w.attend(ctx, [16, 20], [48, 48], 4)
    w.write(ctx, [3, 5], [35, 37])
    w.check_pool()
    b, cu = w.batch([48, 48], [48, 48])
    assert kvc.kvc_validate_batch(w.cache, b, w.table, cu, [48, 48], False) == kvc.KVC_OK
    assert kvc.kvc_validate_batch(w.cache, b, w.table, cu, [48, 48], True) == kvc.KVC_E_DUP_DST
    k, v = (torch.zeros((96, 2, 64), dtype=w.dt, device="cuda") for _ in range(2))
    kvc.kvc_cache_read(ctx, w.cache, b, k, v)
    for got, want in zip((k, v), w.host.read(w.table, cu, [48, 48], 96, w.dt)):
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("rows", [1, 40])
def test_offsets_beyond_32_bits(ctx, rows):
    """Pages 256 MiB apart in pools of 5 GiB, rows 128 MiB apart."""
    w = World("INT8", 1, 128, 16, [70, 200], "bf16", seed=23)
    P, gap = w.host.k.shape[0], 1 << 28
    assert P * gap > 1 << 32
    pools = [torch.zeros(P * gap, dtype=torch.int8, device="cuda") for _ in range(2)]
    k, v, ks, vs = w.dev
    wide_k = pools[0].as_strided((P, 1, 16, 128), (gap, 16 * 128, 128, 1))
    wide_v = pools[1].as_strided((P, 1, 128, 16), (gap, 16 * 128, 16, 1))
    wide_k.copy_(k), wide_v.copy_(v)
    w.dev = (wide_k, wide_v, ks, vs)
    w.cache = kvc.Cache(*w.dev)
    w.write(ctx, [70, 200], [70, 200])
    w.check_pool()
    w.widen(200)
    n = 2 * rows
    far = torch.zeros(n << 26, dtype=torch.bfloat16, device="cuda")
    q = far.as_strided((n, 2, 128), (1 << 26, 128, 1))
    x = w.values(n, 2)
    q.copy_(x)
    b, cu = w.batch([rows, rows], [70, 200])
    o = kvc.Attend(2)
    z = torch.zeros((n, 2), device="cuda")
    ws = torch.zeros(kvc.kvc_plan_attend(w.cache, b, o) + 16, dtype=torch.uint8, device="cuda")
    result = far.as_strided((n, 2, 128), (1 << 26, 128, 1), 512)
    kvc.kvc_cache_attend(ctx, w.cache, b, o, q, result, z, ws)
    want = ref.attend(w.host, w.table, cu, [70, 200], x.float().numpy(), 128 ** -0.5, True, 0)
    w.compare(result, z, *want)
    rk = far.as_strided((n, 1, 128), (1 << 26, 128, 1), 1024)
    rv = far.as_strided((n, 1, 128), (1 << 26, 128, 1), 2048)
    kvc.kvc_cache_read(ctx, w.cache, b, rk, rv)
    for got, exp in zip((rk, rv), w.host.read(w.table, cu, [70, 200], n, torch.bfloat16)):
        assert torch.equal(got.cpu(), exp)


def test_attend_scales_far_apart(ctx):
    """Pages whose values differ by many binades: small ones must not be lost where they are all a row sees."""
    for dtype in ("bf16", "fp16"):
        w = World("FP8_DYNAMIC", 1, 64, 16, [64], dtype, seed=14)
        k, v = w.values(64), w.values(64)
        for i, f in enumerate((1.0, 2.0 ** -11, 0.0, 2.0 ** 10)):
            v[16 * i:16 * i + 16] *= f
            k[16 * i:16 * i + 16] *= (1.0, 2.0 ** -6, 1.0, 0.25)[i]
        w.write(ctx, [64], [64], k, v)
        w.check_pool()
        for last in (16, 32, 48, 64):
            w.attend(ctx, [16], [last], 2, window=16)
            w.attend(ctx, [16], [last], 2)


def test_attend_sharp_and_flat(ctx):
    """Scores that differ by hundreds, and all alike over a long context."""
    w = World("INT8", 1, 64, 16, [3000], "fp16", seed=15)
    w.fill(ctx, [3000])
    w.attend(ctx, [2], [3000], 4, scale=3.0)
    w.attend(ctx, [2], [3000], 4, scale=1e-6)
    w.attend(ctx, [2], [3000], 4, q=torch.zeros(2, 4, 64, dtype=torch.float16))


# ------------------------------------------------------------------ metadata that is wrong on the device
def test_bad_metadata_is_reported_and_not_followed(ctx):
    lengths = [40, 33, 20, 64]
    w = World("INT8", 2, 64, 16, lengths, seed=16)
    w.fill(ctx, lengths)
    good = w.table.copy()
    for table_bad in (-1, w.host.k.shape[0], 0x7FFFFFFF):
        w.table = good.copy()
        w.table[1, 1] = table_bad
        flags = torch.zeros(4, dtype=torch.int32, device="cuda")
        # attention hides the page's 16 positions from sequence 1
        for n, columns in ((2, 0), (20, 0), (20, 200)):
            w.widen(columns)
            flags.zero_()
            b, cu = w.batch([n] * 4, lengths, flags=flags)
            q = w.values(4 * n, 4)
            out, z = torch.zeros((4 * n, 4, 64), dtype=w.dt, device="cuda"), torch.zeros((4 * n, 4), device="cuda")
            o = kvc.Attend(4)
            ws = torch.zeros(kvc.kvc_plan_attend(w.cache, b, o) + 16, dtype=torch.uint8, device="cuda")
            kvc.kvc_cache_attend(ctx, w.cache, b, o, q.cuda(), out, z, ws)
            assert flags.tolist() == [0, 2, 0, 0]
            for s in range(4):
                r = slice(n * s, n * s + n)
                one = ref.attend(w.host, good[s:s + 1], [0, n], lengths[s:s + 1], q[r].float().numpy(), 64 ** -0.5,
                                 True, 0, (1,) if s == 1 else ())
                w.compare(out[r], z[r], *one)
        # reads give zeros there, writes leave everything else alone
        flags.zero_()
        b, cu = w.batch(lengths, lengths, flags=flags)
        k, v = (torch.full((sum(lengths), 2, 64), 7.0, dtype=w.dt, device="cuda") for _ in range(2))
        kvc.kvc_cache_read(ctx, w.cache, b, k, v)
        assert flags.tolist() == [0, 2, 0, 0]
        for got, want in zip((k, v), w.host.read(good, cu, lengths, sum(lengths), w.dt)):
            want[40 + 16:40 + 32] = 0
            assert torch.equal(got.cpu(), want)
        flags.zero_()
        k, v = w.values(sum(lengths)), w.values(sum(lengths))
        kvc.kvc_cache_write(ctx, w.cache, b, k.cuda(), v.cuda())
        was = w.host.k[good[1, 1]].copy(), w.host.v[good[1, 1]].copy(), w.host.ks[good[1, 1]].copy(), w.host.vs[good[1, 1]].copy()
        w.host.write(good, cu, lengths, k.float().numpy(), v.float().numpy())
        w.host.k[good[1, 1]], w.host.v[good[1, 1]], w.host.ks[good[1, 1]], w.host.vs[good[1, 1]] = was
        w.check_pool("bad page")
        assert flags.tolist() == [0, 2, 0, 0]


@pytest.mark.parametrize("direct", [True, False], ids=["direct", "search"])
def test_bad_ranges_skip_their_sequence(ctx, direct):
    lengths = [40, 33, 20, 64, 30]
    w = World("FP8_DYNAMIC", 2, 32, 16, lengths, seed=17)
    w.fill(ctx, lengths)
    n = 20
    # (cu, lengths, flagged): rows beyond n_rows, descending rows, more than max_rows, lengths beyond max_len or negative
    cases = [([0, 2, 4, 6, 8, 21], lengths, [4]), ([0, 2, 5, 4, 8, 10], lengths, [2]), ([-3, 2, 4, 6, 8, 10], lengths, [0]),
             ([0, 2, 4, 6, 16, 18], lengths, [3] if direct else []), ([0, 2, 4, 6, 8, 10], [40, 65, 20, 64, 30], [1]),
             ([0, 2, 4, 6, 8, 10], [40, 33, -1, 64, 30], [2]), ([0, 2, 4, 6, 8, -2147483648], lengths, [4]),
             ([0, 2, 4, 2147483647, 8, 10], lengths, [2, 3])]
    for cu, lens, flagged in cases:
        flags = torch.zeros(5, dtype=torch.int32, device="cuda")
        i32 = [torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda") for x in (w.table, cu, lens)]
        # max_rows 4 makes few units for each sequence; 20 has them found by search
        b = kvc.Batch(*i32, n, 4 if direct else 20, 64, flags)
        k, v = (torch.full((n, 2, 32), 7.0, dtype=w.dt, device="cuda") for _ in range(2))
        kvc.kvc_cache_read(ctx, w.cache, b, k, v)
        assert [i for i in range(5) if flags[i] & 1] == flagged, (cu, lens)
        flags.zero_()
        q = w.values(n, 4)
        out = torch.full((n, 4, 32), 7.0, dtype=w.dt, device="cuda")
        o = kvc.Attend(4)
        ws = torch.zeros(kvc.kvc_plan_attend(w.cache, b, o) + 16, dtype=torch.uint8, device="cuda")
        kvc.kvc_cache_attend(ctx, w.cache, b, o, q.cuda(), out, None, ws)
        assert [i for i in range(5) if flags[i] & 1] == flagged, (cu, lens)
        rows = np.zeros(n, bool)
        for s in range(5):
            if s not in flagged:
                rows[cu[s]:cu[s + 1]] = True
        assert bool((out.cpu()[~rows] == 7.0).all()) and bool((k.cpu()[~rows] == 7.0).all())
        if cu == sorted(cu):                               # an ascending cu leaves the good sequences' results alone
            for s in range(5):
                if s not in flagged:
                    r = slice(cu[s], cu[s + 1])
                    one = ref.attend(w.host, w.table[s:s + 1], [0, cu[s + 1] - cu[s]], lens[s:s + 1], q[r].float().numpy(),
                                     32 ** -0.5, True, 0)
                    w.compare(out[r], None, *one)
        # a write touches no page of a skipped sequence
        before = [t.clone() for t in w.dev]
        x = torch.zeros((n, 2, 32), dtype=w.dt, device="cuda")
        kvc.kvc_cache_write(ctx, w.cache, b, x, x)
        for s in flagged:
            pages = [int(p) for p in w.table[s] if 0 <= p < w.host.k.shape[0]]
            for t, u in zip(w.dev, before):
                assert torch.equal(t.view(torch.uint8)[pages], u.view(torch.uint8)[pages])
        for t, u in zip(w.dev, before):
            t.view(torch.uint8).copy_(u.view(torch.uint8))


# ------------------------------------------------------------------ streams, graphs, and the calls together
def test_other_stream_and_current_device_untouched(ctx):
    w = World("FP8_DYNAMIC", 2, 128, 16, [300, 20], seed=18)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b, cu = w.batch([300, 20], [300, 20])
        k, v = w.values(320), w.values(320)
        kd, vd = k.cuda(), v.cuda()
        torch.cuda._sleep(20_000_000)                      # the calls below must queue behind this
        kvc.kvc_cache_write(ctx, w.cache, b, kd, vd, s.cuda_stream)
        k2, v2 = torch.empty_like(kd), torch.empty_like(vd)
        kvc.kvc_cache_read(ctx, w.cache, b, k2, v2, s.cuda_stream)
    s.synchronize()
    w.host.write(w.table, cu, [300, 20], k.float().numpy(), v.float().numpy())
    w.check_pool()
    for got, want in zip((k2, v2), w.host.read(w.table, cu, [300, 20], 320, w.dt)):
        assert torch.equal(got.cpu(), want)


def test_serving_step_in_a_graph(ctx):
    """Write, attend and read captured once; the lengths, rows and inputs change under the graph.  Two graphs with
    a workspace each run side by side."""
    G, final = 4, [4200, 130, 17]
    w = World("INT8", 2, 64, 16, final, "bf16", seed=19)
    past = [4100, 100, 15]
    w.fill(ctx, past)
    lengths = torch.tensor(past, dtype=torch.int32, device="cuda")
    table = torch.tensor(w.table, dtype=torch.int32, device="cuda")
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    batch = kvc.Batch(table, cu, lengths, 3, 1, 4208)
    o = kvc.Attend(2 * G)
    need = kvc.kvc_plan_attend(w.cache, batch, o)
    assert need > 0
    k, v = (torch.zeros((3, 2, 64), dtype=w.dt, device="cuda") for _ in range(2))
    q = torch.zeros((3, 2 * G, 64), dtype=w.dt, device="cuda")
    sides = []
    for _ in range(2):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        out, z = torch.empty_like(q), torch.empty((3, 2 * G), device="cuda")
        back = torch.empty_like(k), torch.empty_like(v)
        st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=st):
            if not sides:                                  # the first graph writes, both attend and read
                kvc.kvc_cache_write(ctx, w.cache, batch, k, v, st.cuda_stream)
            kvc.kvc_cache_attend(ctx, w.cache, batch, o, q, out, z, ws, st.cuda_stream)
            kvc.kvc_cache_read(ctx, w.cache, batch, *back, st.cuda_stream)
        sides.append((st, graph, out, z, back, ws))
    for step in range(4):
        now = [p + 1 + step for p in past]
        lengths.copy_(torch.tensor(now, dtype=torch.int32))
        kk, vv, qq = w.values(3), w.values(3), w.values(3, 2 * G)
        k.copy_(kk), v.copy_(vv), q.copy_(qq)
        torch.cuda.synchronize()
        sides[0][1].replay()
        torch.cuda.synchronize()
        for i in range(2):                                 # now side by side, the first one's write idempotent
            with torch.cuda.stream(sides[i][0]):
                sides[i][1].replay()
        torch.cuda.synchronize()
        cuh = [0, 1, 2, 3]
        w.host.write(w.table, cuh, now, kk.float().numpy(), vv.float().numpy())
        w.check_pool(f"step {step}")
        want = ref.attend(w.host, w.table, cuh, now, qq.float().numpy(), 64 ** -0.5, True, 0)
        rows = w.host.read(w.table, cuh, now, 3, w.dt)
        eager, ez = torch.empty_like(q), torch.empty((3, 2 * G), device="cuda")
        kvc.kvc_cache_attend(ctx, w.cache, batch, o, q, eager, ez, torch.empty(need, dtype=torch.uint8, device="cuda"))
        for _, _, out, z, back, _ in sides:
            w.compare(out, z, *want)
            assert torch.equal(out, eager) and torch.equal(z, ez)
            assert torch.equal(back[0].cpu(), rows[0]) and torch.equal(back[1].cpu(), rows[1])


def test_restore_attend_and_offload_again(ctx):
    """The library's two caches together: engine pages are decoded from an encoded buffer, brought into the 8-bit
    cache, attended, extended by a token, read back into engine pages and encoded again."""
    H, D, T, pages = 4, 128, 16, 12
    eng_k, eng_v = (torch.randn(pages, T, H, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    lay = kvc.Layout.separate([eng_k], [eng_v], H, D, T)
    codec = kvc.Codec("FP8_DYNAMIC", "INT8", crc=True)
    ids = np.array([7, 2, 9, 4], np.int32)

    def encode(layout, page_ids):
        slot, spill, _ = kvc.kvc_plan(layout, codec, len(page_ids))
        buf = torch.zeros(slot + spill, dtype=torch.uint8, device="cuda")
        desc = torch.zeros(len(page_ids) * 2 * 32, dtype=torch.uint8, device="cuda")
        kvc.kvc_encode_pages(ctx, layout, codec, page_ids, buf.data_ptr(), slot + spill, desc.data_ptr())
        return buf

    buf = encode(lay, ids)
    res_k, res_v = torch.zeros_like(eng_k[:5]), torch.zeros_like(eng_v[:5])
    res = kvc.Layout.separate([res_k], [res_v], H, D, T)
    kvc.kvc_decode_pages(ctx, res, codec, buf.data_ptr(), buf.numel(), np.arange(4, dtype=np.int32))
    w = World("FP8_DYNAMIC", H, D, T, [4 * T + 1], "bf16", seed=20)
    rows_k, rows_v = res_k.view(5 * T, H, D), res_v.view(5 * T, H, D)
    w.write(ctx, [4 * T], [4 * T], rows_k[:4 * T].cpu(), rows_v[:4 * T].cpu())
    w.check_pool("restored")
    w.attend(ctx, [4 * T], [4 * T], 2)
    w.write(ctx, [1], [4 * T + 1])
    w.attend(ctx, [1], [4 * T + 1], 2)
    # back into engine pages: a page pool is a row tensor
    b, cu = w.batch([4 * T + 1], [4 * T + 1])
    kvc.kvc_cache_read(ctx, w.cache, b, rows_k, rows_v)
    torch.cuda.synchronize()
    want = w.host.read(w.table, cu, [4 * T + 1], 4 * T + 1, torch.bfloat16)
    assert torch.equal(rows_k[:4 * T + 1].cpu(), want[0]) and torch.equal(rows_v[:4 * T + 1].cpu(), want[1])
    again = encode(res, np.arange(5, dtype=np.int32))
    out_k, out_v = torch.zeros_like(res_k), torch.zeros_like(res_v)
    kvc.kvc_decode_pages(ctx, kvc.Layout.separate([out_k], [out_v], H, D, T), codec, again.data_ptr(), again.numel(),
                         np.arange(5, dtype=np.int32))
    # each codec is off by half a step of a value's own scale at most: E4M3 2^-4 of it, INT8 amax / 254 (and a bf16 rounding)
    for a, b_, rel, ab in ((out_k, res_k, 2.0 ** -4 + 2.0 ** -8, 448 * 2.0 ** -10 / 448), (out_v, res_v, 2.0 ** -8, 1 / 254)):
        a, b_ = a.float(), b_.float()
        top = b_.abs().amax(3, keepdim=True)
        assert bool(((a - b_).abs() <= rel * b_.abs() + 1.01 * ab * top).all())
