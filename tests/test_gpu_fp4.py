"""The 4-bit cache on the GPU: quantising writes and reads bit for bit, decode within what
rounding allows of the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_315_gb300 as m

    m.build()
    torch.cuda.set_device(0)
    m.pkv_device_error()
    return m


def f64(t):
    return t.double().cpu().numpy()


# ---- writes and reads -------------------------------------------------------------------------


def _rows(n, Hkv, D, dtype, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((n, Hkv, D)) * np.exp(rng.normal(0, 2, (n, Hkv, 1))))
    x = x.to(TORCH[dtype])
    if n >= 8:
        x[0] = 0
        x[1, 0, 3] = float("nan")
        x[2, 0, D - 1] = float("-inf")
        x[3] = torch.finfo(TORCH[dtype]).max                # bf16: the scale stays finite
        x[4] *= 0
        x[4, :, 5] = -torch.finfo(TORCH[dtype]).tiny * 2 ** -6  # a subnormal
        # ties: amax 6 gives scale 1, and these are halfway between two codes
        x[5] = 0
        x[5, :, :16] = torch.tensor([6, 5, -5, 3.5, 2.5, 1.75, 1.25, .75, .25, -.25, -.75, -1.25,
                                     -2.5, 4.5, 5.5, -6]).to(x.dtype)
        x[6] = x[5] * 1.25
        x[7] = -0.0
    return x


@pytest.mark.parametrize("dtype,Hkv,D,bs,n", [
    ("bf16", 8, 128, 16, 37), ("f16", 3, 128, 32, 64), ("f32", 1, 128, 64, 9), ("f32", 5, 64, 16, 30),
    ("bf16", 2, 256, 16, 20), ("f16", 7, 32, 16, 41), ("bf16", 40, 128, 1, 11), ("f16", 1, 64, 5, 1),
    ("bf16", 1, 32, 3, 2), ("f32", 2, 256, 16, 700)])
def test_write_then_read_bit_exact(pkv, dtype, Hkv, D, bs, n):
    NB = -(-n // bs) + 3
    rng = np.random.default_rng(n)
    slots = rng.choice(NB * bs, n, replace=False)
    if n > 10:
        slots[[n - 1, n // 2]] = -1, -(2 ** 40)
    x, y = _rows(n, Hkv, D, dtype, 1), _rows(n, Hkv, D, dtype, 2)
    caches = [torch.full((NB, bs, Hkv, D // 2), 0xA5, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.full((NB, Hkv, bs), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    sm = torch.from_numpy(slots).cuda()
    pkv.kv_cache_write_fp4(x.cuda(), y.cuda(), *caches, *scales, sm)
    assert pkv.pkv_device_error() == 0
    live = slots >= 0
    for src, cache, scale in zip((x, y), caches, scales):
        code, s = ref.encode_rows(f64(src))
        want_c = np.full((NB * bs, Hkv, D // 2), 0xA5, np.uint8)
        want_s = np.full((NB * bs, Hkv), 3.0)
        want_c[slots[live]] = ref.pack(code)[live]
        want_s[slots[live]] = s[live]
        assert np.array_equal(cache.cpu().numpy().reshape(NB * bs, Hkv, D // 2), want_c)
        assert np.array_equal(f64(scale).transpose(0, 2, 1).reshape(NB * bs, Hkv), want_s,
                              equal_nan=True)
    for out in ("bf16", "f16", "f32"):
        got = [torch.full((n, Hkv, D), 7.0, dtype=TORCH[out], device="cuda") for _ in "kv"]
        pkv.kv_cache_read_fp4(*got, *caches, *scales, sm)
        assert pkv.pkv_device_error() == 0
        for g, cache, scale in zip(got, caches, scales):
            v = ref.values(cache.cpu().numpy().reshape(NB * bs, Hkv, D // 2)[np.abs(slots) % (NB * bs)],
                           f64(scale).transpose(0, 2, 1).reshape(NB * bs, Hkv)[np.abs(slots) % (NB * bs)])
            want = torch.from_numpy(v).float().to(TORCH[out]).double().numpy()
            want[~live] = 7.0
            assert np.array_equal(f64(g), want, equal_nan=True)


def test_reads_repeat_slots_and_skip_those_out_of_range(pkv):
    NB, bs, Hkv, D, n = 3, 16, 2, 128, 6
    x = _rows(n, Hkv, D, "bf16", 3)
    caches = [torch.zeros((NB, bs, Hkv, D // 2), dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.zeros((NB, Hkv, bs), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    before = [t.clone() for t in caches + scales]
    pkv.kv_cache_write_fp4(x.cuda(), x.cuda(), *caches, *scales,
                           torch.tensor([48, -1, 2 ** 40, 49, 5, -9]).cuda())
    assert pkv.pkv_device_error() == pkv.PKV_DERR_SLOT
    changed = torch.zeros(NB, bs, dtype=torch.bool)
    changed[0, 5] = True
    for t, b in zip(caches, before):
        assert torch.equal((t != b).flatten(2).any(-1).cpu(), changed)
    got = [torch.full((n, Hkv, D), 7.0, device="cuda") for _ in "kv"]
    pkv.kv_cache_read_fp4(*got, *caches, *scales, torch.tensor([5, 5, 48, -1, 5, 2 ** 62]).cuda())
    assert pkv.pkv_device_error() == pkv.PKV_DERR_SLOT
    code, s = ref.encode_rows(f64(x[4]))
    want = ref.values(ref.pack(code), s)
    for i in (0, 1, 4):
        assert np.array_equal(f64(got[0][i]), want)
    assert (got[0][[2, 3, 5]] == 7).all()


# ---- decode -----------------------------------------------------------------------------------


class Case:
    """A batch over a 4-bit cache with shuffled blocks; everything dead is NaN scales and ids
    far out of range."""

    def __init__(self, dtype, Hq, Hkv, D, bs, lens, seed=1, q_scale=1.0, scale=None, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.lens, self.bs = dtype, np.asarray(lens), bs
        B = len(lens)
        used = [-(-int(n) // bs) for n in lens]
        MB = max(1, max(used)) + 1
        NB = sum(used) + 3
        ids = torch.randperm(NB, generator=g)
        self.tables = np.full((B, MB), 2 ** 30, np.int32)
        at = 0
        for s, u in enumerate(used):
            self.tables[s, :u] = ids[at:at + u].numpy()
            at += u
        self.q = (torch.randn(B, Hq, D, generator=g) * q_scale).to(TORCH[dtype])
        self.scale = 1 / math.sqrt(D) if scale is None else scale
        self.kc, self.vc = (torch.randint(0, 256, (NB, bs, Hkv, D // 2), generator=g).to(torch.uint8)
                            for _ in "kv")
        self.ks, self.vs = ((0.3 * torch.exp(spread * torch.randn(NB, Hkv, bs, generator=g))).bfloat16()
                            for _ in "kv")
        live = torch.zeros(NB, bs, dtype=torch.bool)
        for s, n in enumerate(lens):
            for p in range(int(n)):
                live[self.tables[s, p // bs], p % bs] = True
        for t in (self.ks, self.vs):
            t.transpose(1, 2)[~live] = float("nan")

    def dev(self):
        return [t.cuda() for t in (self.kc, self.vc, self.ks, self.vs)] + [
            torch.from_numpy(self.tables).cuda(), torch.from_numpy(self.lens.astype(np.int32)).cuda()]

    def run(self, pkv, **kw):
        q = self.q.cuda()
        out = torch.full_like(q, 9.0)
        pkv.paged_attn_decode_fp4(out, q, *self.dev(), self.scale, **kw)
        return out

    def check(self, got):
        want = ref.decode(f64(self.q), self.kc.numpy(), self.vc.numpy(), f64(self.ks), f64(self.vs),
                          self.tables, self.lens, self.scale)
        tol = ref.decode_tolerance(self.dtype, self.lens, self.q.shape[2], *want)
        err = np.abs(f64(got) - want[0])
        assert np.isfinite(f64(got)).all()
        worst = np.unravel_index(np.argmax(err - tol), err.shape)
        assert (err <= tol).all(), (worst, err[worst], tol[worst], want[0][worst])
        assert (f64(got)[self.lens == 0] == 0).all()


LENS = [0, 1, 15, 16, 17, 127, 128, 129, 300, 1111, 0, 64]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [
    (4, 4, 128, 16), (8, 1, 128, 16), (6, 2, 128, 32), (16, 2, 128, 64), (2, 1, 128, 16),
    (5, 1, 128, 16), (16, 1, 128, 32), (12, 1, 128, 16), (9, 1, 128, 16), (14, 2, 128, 16),
    (4, 2, 64, 16), (8, 1, 64, 32), (4, 1, 32, 16), (3, 3, 256, 16), (8, 2, 128, 1), (4, 2, 128, 48),
    (8, 2, 128, 8), (8, 1, 128, 128)])
def test_decode_shapes(pkv, dtype, Hq, Hkv, D, bs):
    c = Case(dtype, Hq, Hkv, D, bs, LENS, seed=Hq + D + bs)
    got = c.run(pkv)
    assert pkv.pkv_device_error() == 0
    c.check(got)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", [[1], [2], [33], [5000], [128] * 70, [1, 4096, 1, 2000, 0, 3],
                                  [0, 0, 0], [257] * 9 + [0]])
def test_decode_batches(pkv, dtype, lens):
    c = Case(dtype, 8, 2, 128, 16, lens, seed=len(lens))
    got = c.run(pkv)
    assert pkv.pkv_device_error() == 0
    c.check(got)


def test_decode_many_sequences(pkv):
    c = Case("bf16", 2, 2, 128, 16, np.arange(700) % 23, seed=4)
    c.check(c.run(pkv))
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("q_scale,scale,spread", [
    (300.0, None, 1.0),       # one token takes all of the weight
    (1.0, 0.0, 1.0),          # every token weighs the same
    (1.0, -0.1, 1.0),
    (2.0 ** -12, 30.0, 1.0),  # small queries, among fp16's subnormals
    (1.0, None, 4.0)])        # row scales over many orders of magnitude
def test_decode_ranges(pkv, dtype, q_scale, scale, spread):
    c = Case(dtype, 8, 2, 128, 16, [1, 40, 700, 129], seed=11, q_scale=q_scale, scale=scale,
             spread=spread)
    got = c.run(pkv)
    assert pkv.pkv_device_error() == 0
    c.check(got)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_decode_sink_token(pkv, dtype):
    """One key far above the others, whose many small weights together still count."""
    c = Case(dtype, 4, 1, 128, 16, [4000, 900], seed=5, spread=0.0)
    c.ks[:] = torch.where(torch.isnan(c.ks), c.ks, torch.tensor(0.02).bfloat16())
    row = c.tables[0, 3]
    c.kc[row, 7, 0] = 0x77          # all 6
    c.ks[row, 0, 7] = 0.25
    c.q = c.q.abs()                 # score of the sink: about 0.8 * 6 * 0.25 * sqrt(128) = 13.6
    c.vs[row, 0, 7] = 0.001         # and its value is small, so the others decide the output
    c.check(c.run(pkv))


def test_decode_non_finite_rows(pkv):
    """A NaN row reaches the sequences and heads that attend it, and no others; queries that
    are not finite reach their own head."""
    for dtype in ("bf16", "f16", "f32"):
        c = Case(dtype, 8, 2, 128, 16, [40, 300, 129], seed=6)
        clean = c.run(pkv)
        c.vs[c.tables[1, 3], 1, 2] = float("nan")
        c.ks[c.tables[2, 8], 0, 0] = float("nan")   # its last token, alone in its tile
        got = f64(c.run(pkv))
        bad = np.isnan(got)
        want = np.zeros_like(bad)
        want[1, 4:] = True
        want[2, :4] = True
        assert np.array_equal(bad, want)
        assert np.array_equal(got[~want], f64(clean)[~want])
        c = Case(dtype, 8, 2, 128, 16, [40, 300, 129], seed=6)
        c.q[1, 5, 100] = float("nan")
        c.q[2, 0, 0] = float("inf")
        bad = np.isnan(f64(c.run(pkv)))
        assert bad[1, 5].all() and bad[2, 0].all() and bad.sum() == 2 * 128


@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("f32", 16), ("f16", 64)])
def test_decode_bad_ids_and_lengths(pkv, dtype, bs):
    c = Case(dtype, 8, 2, 128, bs, [40, 300, 129, 64], seed=7)
    c.kc = torch.cat([c.kc, torch.zeros_like(c.kc[:1])])
    c.vc = torch.cat([c.vc, torch.zeros_like(c.vc[:1])])
    c.ks = torch.cat([c.ks, torch.ones_like(c.ks[:1])])
    c.vs = torch.cat([c.vs, torch.ones_like(c.vs[:1])])
    zero = c.kc.shape[0] - 1
    for bad in (-1, zero + 1, 2 ** 30, -(2 ** 31)):
        c.tables[1, 2] = bad
        got = c.run(pkv)
        assert pkv.pkv_device_error() == pkv.PKV_DERR_BLOCK_ID
        c.tables[1, 2] = zero          # reads as zeros: keys 0 and values 0
        c.check(got)
        assert torch.equal(got, c.run(pkv))
    cap = c.tables.shape[1] * bs
    lens = c.lens.copy()
    c.tables[0, :] = zero
    c.lens = np.array([cap + 5, 300, -7, 64])
    got = c.run(pkv)
    assert pkv.pkv_device_error() == pkv.PKV_DERR_CONTEXT
    c.lens = np.array([cap, 300, 0, 64])
    c.check(got)
    c.lens = lens


def test_decode_does_not_depend_on_block_order_or_schedule(pkv):
    c = Case("bf16", 8, 2, 128, 16, [700, 1, 300, 2000], seed=8)
    first = c.run(pkv)
    for _ in range(3):
        assert torch.equal(c.run(pkv), first)
    NB = c.kc.shape[0]
    perm = torch.randperm(NB, generator=torch.Generator().manual_seed(1))
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(NB)
    for n in ("kc", "vc", "ks", "vs"):
        setattr(c, n, getattr(c, n)[perm])
    live = c.tables < NB
    c.tables[live] = inv.numpy()[c.tables[live]]
    assert torch.equal(c.run(pkv), first)


def test_decode_offsets_past_32_bits(pkv):
    """A cache of more than 2^32 bytes: the blocks in use lie at its two ends."""
    Hkv, D, bs = 8, 128, 16
    NB = (2 ** 32 + 2 ** 28) // (bs * Hkv * D // 2)
    lens = [70, 200]
    c = Case("bf16", 16, Hkv, D, bs, lens, seed=9)
    far = np.concatenate([np.arange(NB - c.kc.shape[0] + 3, NB), np.arange(3)])
    kc, vc = (torch.zeros(NB, bs, Hkv, D // 2, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(NB, Hkv, bs, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    at = torch.from_numpy(far).cuda()
    for big, small in ((kc, c.kc), (vc, c.vc), (ks, c.ks), (vs, c.vs)):
        big[at] = small.cuda()
    table = c.tables.copy()
    live = table < 2 ** 30
    table[live] = far[table[live]]
    q = c.q.cuda()
    out = torch.empty_like(q)
    pkv.paged_attn_decode_fp4(out, q, kc, vc, ks, vs, torch.from_numpy(table).cuda(),
                              torch.from_numpy(c.lens.astype(np.int32)).cuda(), c.scale)
    assert pkv.pkv_device_error() == 0
    c.check(out)
    # rows written and read at the far end
    x = _rows(9, Hkv, D, "bf16", 5).cuda()
    slots = torch.arange(NB * bs - 9, NB * bs).cuda()
    pkv.kv_cache_write_fp4(x, x, kc, vc, ks, vs, slots)
    a, b = torch.empty_like(x), torch.empty_like(x)
    pkv.kv_cache_read_fp4(a, b, kc, vc, ks, vs, slots)
    assert pkv.pkv_device_error() == 0
    code, s = ref.encode_rows(f64(x))
    want = torch.from_numpy(ref.values(ref.pack(code), s)).float().bfloat16()
    assert np.array_equal(f64(a), f64(want), equal_nan=True) and torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_decode_workspace(pkv):
    c = Case("bf16", 8, 2, 128, 16, [700, 1, 300, 2000], seed=8)
    first = c.run(pkv)
    need = pkv.paged_attn_decode_fp4_workspace_size(4, 8, 2, 128, 16, c.tables.shape[1])
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.run(pkv, workspace=ws), first)
    with pytest.raises(pkv.PagedKVError) as e:
        c.run(pkv, workspace=ws[:-16])
    assert e.value.code == -2


def test_decode_streams_and_graphs(pkv):
    """Two calls on two streams at once, and two captured graphs replayed in turn with new
    lengths and queries in the same buffers."""
    cases = [Case("bf16", 8, 2, 128, 16, [700, 1, 300, 2000], seed=8),
             Case("bf16", 8, 2, 128, 16, [3000, 5, 0, 40], seed=12)]
    want = [c.run(pkv) for c in cases]
    torch.cuda.synchronize()
    state = [(c.q.cuda(), c.dev()) for c in cases]
    outs = [torch.full_like(s[0], 9.0) for s in state]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, (q, args), out, st in zip(cases, state, outs, streams):
            pkv.paged_attn_decode_fp4(out, q, *args, c.scale, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    graphs = []
    for c, (q, args), out in zip(cases, state, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_attn_decode_fp4(out, q, *args, c.scale)
        graphs.append(g)
    for o in outs:
        o.fill_(9.0)
    for i in (0, 1, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    # other lengths in the same buffers
    c, (q, args) = cases[0], state[0]
    args[5].copy_(torch.tensor([17, 0, 299, 1500], dtype=torch.int32))
    c.lens = np.array([17, 0, 299, 1500])
    graphs[0].replay()
    torch.cuda.synchronize()
    c.check(outs[0])


def test_decode_on_given_streams(pkv):
    """The default stream by object and by handle, and a captured stream given by name."""
    c = Case("bf16", 8, 2, 128, 16, [700, 1, 300, 2000], seed=8)
    want = c.run(pkv)
    torch.cuda.synchronize()
    assert torch.equal(c.run(pkv, stream=torch.cuda.default_stream()), want)
    assert torch.equal(c.run(pkv, stream=0), want)
    q, args = c.q.cuda(), c.dev()
    out = torch.full_like(q, 9.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pkv.paged_attn_decode_fp4(out, q, *args, c.scale, stream=side)
    for _ in range(3):
        c.run(pkv)  # eager calls between the replays
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_decode_scales_off_16_bytes(pkv, dtype):
    c = Case(dtype, 8, 2, 128, 16, [700, 1, 0, 300, 2000], seed=8)
    args = c.dev()
    for i in (2, 3):
        flat = torch.empty(args[i].numel() + 1, dtype=torch.bfloat16, device="cuda")
        flat[1:] = args[i].flatten()
        args[i] = flat[1:].view(args[i].shape)
        assert args[i].data_ptr() % 16 != 0
    out = torch.full_like(c.q, 9.0, device="cuda")
    pkv.paged_attn_decode_fp4(out, c.q.cuda(), *args, c.scale)
    assert pkv.pkv_device_error() == 0
    c.check(out)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,bs", [("f16", 16, 2, 128, 16), ("bf16", 2, 1, 64, 16),
                                               ("f32", 6, 1, 128, 32), ("bf16", 3, 1, 128, 16)])
def test_decode_more_tiles_than_ranges(pkv, dtype, Hq, Hkv, D, bs):
    c = Case(dtype, Hq, Hkv, D, bs, [60000, 17, 0, 70000, 129, 128], seed=21)
    got = c.run(pkv)
    assert pkv.pkv_device_error() == 0
    c.check(got)


@pytest.mark.parametrize("order", ["mixed", "rising", "falling"])
@pytest.mark.parametrize("dtype,Hq,Hkv,D", [("bf16", 40, 40, 128), ("bf16", 96, 16, 128),
                                            ("f16", 64, 8, 128), ("bf16", 16, 16, 64),
                                            ("f32", 32, 16, 32)])
def test_decode_ranges_of_many_short_sequences(pkv, dtype, Hq, Hkv, D, order):
    """More than four tiles to a range, where a sequence's start counts beside its tiles."""
    lens = np.arange(240) * 37 % 450
    lens[::17] = 0
    if order != "mixed":
        lens = np.sort(lens)[::1 if order == "rising" else -1].copy()
    c = Case(dtype, Hq, Hkv, D, 16, lens, seed=D + Hq)
    got = c.run(pkv)
    assert pkv.pkv_device_error() == 0
    c.check(got)


# ---- together ---------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype,Hq,Hkv,D,bs", [("bf16", 8, 2, 128, 16), ("f16", 3, 1, 128, 32),
                                               ("bf16", 4, 2, 64, 16)])
def test_serving_steps(pkv, dtype, Hq, Hkv, D, bs):
    """Prompts, decode steps, a finished request and a new one: tables and slots from
    kv_resize_requests, rows quantised into them, decode over what was written, against the
    same steps on plain arrays; the context read back feeds chunked prefill."""
    B, MB = 4, 12
    NB = 20
    rng = np.random.default_rng(3)
    dev = dict(tables=torch.zeros(B, MB, dtype=torch.int32, device="cuda"),
               lens=torch.zeros(B, dtype=torch.int32, device="cuda"),
               ring=torch.arange(NB, dtype=torch.int32, device="cuda"),
               pool=torch.tensor([0, NB, 0, 0], dtype=torch.int32, device="cuda"))
    kc, vc = (torch.zeros(NB, bs, Hkv, D // 2, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(NB, Hkv, bs, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    history = [[np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))] for _ in range(B)]
    lens = [0] * B
    for target in ([33, 16, 1, 0], [34, 17, 2, 70], [35, 0, 3, 71], [36, 5, 4, 72], [20, 6, 5, 73]):
        rows = sum(max(0, n - o) for n, o in zip(target, lens))
        slots = torch.empty(rows + 2, dtype=torch.int64, device="cuda")
        pkv.kv_resize_requests(dev["tables"], dev["lens"],
                               torch.tensor(target, dtype=torch.int32, device="cuda"), dev["ring"],
                               dev["pool"], slots, None, bs, NB)
        x = [torch.from_numpy(rng.standard_normal((rows + 2, Hkv, D))).to(TORCH[dtype]) for _ in "kv"]
        pkv.kv_cache_write_fp4(x[0].cuda(), x[1].cuda(), kc, vc, ks, vs, slots)
        at = 0
        for s in range(B):
            n = max(0, target[s] - lens[s])
            for i in (0, 1):
                code, sc = ref.encode_rows(f64(x[i][at:at + n]))
                history[s][i] = np.concatenate([history[s][i], ref.values(ref.pack(code), sc)])[:target[s]]
            at += n
        lens = target
        q = torch.from_numpy(rng.standard_normal((B, Hq, D))).to(TORCH[dtype])
        out = torch.empty_like(q.cuda())
        pkv.paged_attn_decode_fp4(out, q.cuda(), kc, vc, ks, vs, dev["tables"], dev["lens"],
                                  1 / math.sqrt(D))
        assert pkv.pkv_device_error() == 0
        assert dev["lens"].tolist() == target
        tables = dev["tables"].cpu().numpy()
        want = ref.decode(f64(q), kc.cpu().numpy(), vc.cpu().numpy(), f64(ks), f64(vs), tables,
                          target, 1 / math.sqrt(D))
        assert (np.abs(f64(out) - want[0]) <= ref.decode_tolerance(dtype, target, D, *want)).all()
        for s in range(B):  # what the tables name is what was written
            pos = np.arange(target[s])
            sl = torch.from_numpy(tables[s, pos // bs].astype(np.int64) * bs + pos % bs).cuda()
            k = torch.empty(len(pos), Hkv, D, device="cuda")
            v = torch.empty_like(k)
            pkv.kv_cache_read_fp4(k, v, kc, vc, ks, vs, sl)
            assert np.array_equal(f64(k), history[s][0]) and np.array_equal(f64(v), history[s][1])
    # request 3's context in 16 bits, and the last 3 of its tokens as a prefill chunk over it
    n = lens[3]
    pad = -(-n // bs) * bs
    pos = np.arange(pad)
    sl = tables[3, pos // bs].astype(np.int64) * bs + pos % bs
    sl[n:] = -1
    k, v = (torch.zeros(pad, Hkv, D, dtype=TORCH[dtype], device="cuda") for _ in "kv")
    pkv.kv_cache_read_fp4(k, v, kc, vc, ks, vs, torch.from_numpy(sl).cuda())
    q = torch.from_numpy(rng.standard_normal((3, Hq, D))).to(TORCH[dtype])
    out = torch.empty_like(q.cuda())
    pkv.paged_attn_prefill(out, q.cuda(), k.view(-1, bs, Hkv, D), v.view(-1, bs, Hkv, D),
                           torch.arange(pad // bs, dtype=torch.int32, device="cuda").view(1, -1),
                           torch.tensor([n], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, 3], dtype=torch.int32, device="cuda"), 3, 1 / math.sqrt(D))
    assert pkv.pkv_device_error() == 0
    kh, vh = f64(k), f64(v)
    for i in range(3):
        for h in range(Hq):
            m = n - 2 + i
            z = kh[:m, h * Hkv // Hq] @ f64(q)[i, h] / math.sqrt(D)
            w = np.exp(z - z.max())
            want = w / w.sum() @ vh[:m, h * Hkv // Hq]
            # the weights and the output are rounded to the element type
            half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
            bound = (w / w.sum()) @ np.abs(vh[:m, h * Hkv // Hq])
            assert (np.abs(f64(out)[i, h] - want) <= 2.5 * half * bound + half * np.abs(want)).all()
