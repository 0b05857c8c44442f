"""The 4-bit cache and request-resize entry points without a GPU: argument checks, sizes, and
the plain implementations that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_reference as ref


@pytest.fixture(scope="module")
def lib():
    import paged_kv_cache_315_gb300 as pkv

    pkv.build()
    return pkv.load()


NULL = None


def _decode(lib, B=2, Hq=8, Hkv=2, D=128, bs=16, MB=4, NB=8, dt=1, ptr=NULL, ws=NULL, wsb=0):
    return lib.paged_attn_decode_fp4(ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, B, Hq, Hkv, D, bs, MB,
                                     NB, 0.1, dt, ws, wsb, NULL)


def test_decode_refusals(lib):
    assert _decode(lib) == -1                                  # null pointers
    assert _decode(lib, B=0) == 0
    assert _decode(lib, B=-1) == -1
    assert _decode(lib, Hq=6, Hkv=4) == -1
    assert _decode(lib, dt=3) == -1
    assert _decode(lib, D=96) == -4
    assert _decode(lib, D=512) == -4
    assert _decode(lib, bs=0) == -1
    assert _decode(lib, bs=2**16, MB=2**15) == -1              # lengths past 32 bits
    assert _decode(lib, bs=2**16, NB=2**15) == -1
    # misaligned pointers are found before any device work
    assert _decode(lib, ptr=ctypes.c_void_p(4096 + 8)) == -1
    assert _decode(lib, ptr=ctypes.c_void_p(4096 + 16)) == -1  # the codes want 32 bytes


def test_row_refusals(lib):
    def rows(fn, n=2, Hkv=2, D=128, bs=16, NB=8, dt=1, ptr=NULL):
        return fn(ptr, ptr, ptr, ptr, ptr, ptr, ptr, n, Hkv, D, bs, NB, dt, NULL)

    for fn in (lib.kv_cache_write_fp4, lib.kv_cache_read_fp4):
        assert rows(fn) == -1
        assert rows(fn, n=0) == 0
        assert rows(fn, n=-1) == -1
        assert rows(fn, Hkv=0) == -1
        assert rows(fn, D=48) == -4
        assert rows(fn, dt=9) == -1
        assert rows(fn, ptr=ctypes.c_void_p(4096 + 8)) == -1


def test_resize_refusals(lib):
    def resize(B=2, rows=4, ring=8, bs=16, MB=4, NB=8, ptr=NULL, ws=NULL, wsb=0):
        return lib.kv_resize_requests(ptr, ptr, ptr, ptr, ptr, ptr, ptr, B, rows, ring, bs, MB, NB,
                                      ws, wsb, NULL)

    assert resize() == -1
    assert resize(B=0, rows=0) == 0
    assert resize(B=-1) == -1
    assert resize(ring=0) == -1
    assert resize(MB=2**27) == -1
    assert resize(B=2**20, MB=2**12) == -1
    ok = ctypes.c_void_p(4096)
    assert resize(ptr=ok) == -2                                # no workspace
    assert resize(ptr=ok, ws=ok, wsb=8) == -2
    assert resize(ptr=ctypes.c_void_p(4098), ws=ok, wsb=1 << 20) == -1


def test_sizes_and_names(lib):
    import paged_kv_cache_315_gb300 as pkv

    size = pkv.paged_attn_decode_fp4_workspace_size
    assert size(1, 8, 8, 128, 16, 8) == 0                      # one 128-token tile: never split
    assert size(1, 8, 8, 128, 16, 9) > 0
    assert size(1, 8, 3, 128, 16, 9) == 0                      # not a shape
    # 57 ranges of 8 units on 456 places: two partials for each, row by row
    assert size(32, 32, 8, 128, 16, 2048) >= 57 * 2 * 32 * (128 + 2) * 4
    assert size(4, 1024, 1024, 128, 16, 2048) == 0             # more units than places: no split
    assert pkv.kv_resize_requests_workspace_size(0) == 0
    assert pkv.kv_resize_requests_workspace_size(100) >= 4 * 400
    assert "pool" in pkv.pkv_strerror(pkv.PKV_DERR_POOL)


def _cache(NB=4, bs=16, Hkv=2, D=128):
    codes = torch.zeros(NB, bs, Hkv, D // 2, dtype=torch.uint8)
    scales = torch.zeros(NB, Hkv, bs, dtype=torch.bfloat16)
    return codes, codes.clone(), scales, scales.clone()


def test_binding_checks_shapes_and_types(monkeypatch):
    import paged_kv_cache_315_gb300 as pkv

    kc, vc, ks, vs = _cache()
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    bt, cl = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(TypeError, match="CUDA"):
        pkv.paged_attn_decode_fp4(q, q, kc, vc, ks, vs, bt, cl, 0.1)
    with pytest.raises(TypeError, match="uint8"):
        pkv.paged_attn_decode_fp4(q, q, kc.float(), vc, ks, vs, bt, cl, 0.1)
    with pytest.raises(TypeError, match="bfloat16"):
        pkv.paged_attn_decode_fp4(q, q, kc, vc, ks.float(), vs, bt, cl, 0.1)
    with pytest.raises(ValueError, match="NB, Hkv, bs"):
        pkv.paged_attn_decode_fp4(q, q, kc, vc, ks.transpose(1, 2), vs, bt, cl, 0.1)
    with pytest.raises(TypeError, match="int32"):
        pkv.paged_attn_decode_fp4(q, q, kc, vc, ks, vs, bt.long(), cl, 0.1)
    with pytest.raises(ValueError, match="shape mismatch"):
        pkv.paged_attn_decode_fp4(q[..., :64], q[..., :64], kc, vc, ks, vs, bt, cl, 0.1)
    with pytest.raises(TypeError, match="one element type"):
        pkv.paged_attn_decode_fp4(q, q.half(), kc, vc, ks, vs, bt, cl, 0.1)
    with pytest.raises(TypeError, match="element type"):
        pkv.paged_attn_decode_fp4(q.double(), q.double(), kc, vc, ks, vs, bt, cl, 0.1)
    k = torch.zeros(3, 2, 128)
    with pytest.raises(TypeError, match="int64"):
        pkv.kv_cache_write_fp4(k, k, kc, vc, ks, vs, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="matching the cache"):
        pkv.kv_cache_read_fp4(k[:, :1], k[:, :1], kc, vc, ks, vs, torch.zeros(3).long())
    with pytest.raises(TypeError, match="CUDA"):
        pkv.kv_cache_write_fp4(k, k, kc, vc, ks, vs, torch.zeros(3).long())
    pkv.kv_cache_write_fp4(k[:0], k[:0], kc, vc, ks, vs, torch.zeros(0).long())  # nothing to do
    state = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        pkv.kv_resize_requests(bt, cl, cl, cl, state, torch.zeros(3).long(), None, 16, 4)
    with pytest.raises(ValueError, match="pool_state"):
        pkv.kv_resize_requests(bt, cl, cl, cl, cl, torch.zeros(3).long(), None, 16, 4)
    with pytest.raises(ValueError, match="query_start"):
        pkv.kv_resize_requests(bt, cl, cl, cl, state, torch.zeros(3).long(), cl, 16, 4)


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    from paged_kv_cache_315_gb300 import _binding

    class Elsewhere(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = torch.zeros(2).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="device 1"):
        _binding._on_current("q", (t,))


# ---- the plain implementations ----------------------------------------------------------------


def test_reference_codes():
    x = np.zeros((1, 16))
    x[0, :15] = [6, -6, 5, 5.01, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, 0.26, -1.75, 1.0, -0.0]
    code, scale = ref.encode_rows(x)
    assert scale[0] == 1.0
    # ties go to the even code: 5 -> 4, 3.5 -> 4, 2.5 -> 2, 1.75 -> 2, 1.25 -> 1, 0.75 -> 1, 0.25 -> 0
    assert code[0].tolist() == [7, 15, 6, 7, 6, 4, 4, 2, 2, 0, 8, 1, 12, 2, 8, 0]
    back = ref.values(ref.pack(code), scale)
    assert back[0, :5].tolist() == [6, -6, 4, 6, 4]
    code, scale = ref.encode_rows(np.array([[np.nan, 1.0], [np.inf, 1.0], [0.0, 0.0], [7.5, -1.25]]))
    assert np.isnan(scale[:2]).all() and scale[2] == 0 and scale[3] == 1.25
    assert code.tolist() == [[0, 0], [0, 0], [0, 0], [7, 10]]


def test_reference_scale_is_the_bf16_nearest():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 32)).astype(np.float32)
    _, scale = ref.encode_rows(x)
    t = (torch.from_numpy(np.abs(x).max(-1)) / torch.tensor(6.0)).bfloat16()
    assert np.array_equal(scale, t.double().numpy())


def test_reference_resize_walk():
    """A pool of 8 blocks of 4 tokens: growth, refusal in order, release and reuse."""
    tables = np.full((3, 4), -7, np.int32)
    lens = np.array([0, 0, 0], np.int32)
    ring = np.arange(8, dtype=np.int32)
    pool = np.array([0, 8, 0, 0], np.int32)
    slots, start, err = ref.resize(tables, lens, [5, 0, 9], ring, pool, 16, 4, 8)
    assert err == 0 and start.tolist() == [0, 5, 5, 14]
    assert slots.tolist() == [0, 1, 2, 3, 4, 8, 9, 10, 11, 12, 13, 14, 15, 16, -1, -1]
    assert tables.tolist() == [[0, 1, -7, -7], [-7] * 4, [2, 3, 4, -7]] and pool[:2].tolist() == [5, 3]
    # request 1 wants four blocks of three: refused; request 2's token fits its last block, and
    # request 0 gives its blocks back
    slots, start, err = ref.resize(tables, lens, [0, 16, 10], ring, pool, 20, 4, 8)
    assert err == 32 and start.tolist() == [0, 0, 16, 17]
    assert slots.tolist() == [-1] * 16 + [17] + [-1] * 3
    assert lens.tolist() == [0, 0, 10] and pool[:2].tolist() == [5, 5]
    free = [int(ring[(pool[0] + i) % 8]) for i in range(pool[1])]
    assert free == [5, 6, 7, 0, 1]
    slots, start, err = ref.resize(tables, lens, [0, 16, 10], ring, pool, 16, 4, 8)
    assert err == 0 and tables[1].tolist() == [5, 6, 7, 0] and pool[:2].tolist() == [1, 1]
