"""Plain implementations of the 4-bit cache operators and of the request resize, in 64 bits
and Python integers, for the tests (no code of the package)."""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_round(x):
    """float64 (fp32 values) -> nearest bf16, ties to even, as float64."""
    with np.errstate(over="ignore"):
        bits = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    bits = (bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000
    return bits.astype(np.uint32).view(np.float32).astype(np.float64)


def encode_rows(x):
    """Rows [..., D] (float64 of any element type's values) -> codes [..., D] (0..15) and
    scales [...] (float64 values of bf16)."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(-1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(x), x, 0.0)).max(-1))
    scale = bf16_round(np.float32(amax) / np.float32(6.0))
    with np.errstate(divide="ignore", invalid="ignore", under="ignore"):
        y = (x.astype(np.float32) / scale[..., None].astype(np.float32)).astype(np.float64)
    y = np.where((scale[..., None] > 0) & ~bad[..., None], y, 0.0)
    dist = np.abs(np.minimum(np.abs(y), 6.0)[..., None] - MAGNITUDES)
    best = dist.min(-1, keepdims=True)
    near = dist == best  # one code, or two equally near neighbours: the even one
    first = near.argmax(-1)
    last = 7 - near[..., ::-1].argmax(-1)
    code = np.where(first % 2 == 0, first, last)
    code = code + 8 * (np.signbit(y) & (scale[..., None] > 0))
    return code.astype(np.uint8), np.where(bad, np.nan, scale)


def pack(codes):
    """Codes [..., D] -> bytes [..., D / 2], the even element in the low half."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def values(packed, scales):
    """float64 values of bytes [..., D / 2] and scales [...]."""
    code = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], 2 * packed.shape[-1])
    v = MAGNITUDES[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.asarray(scales, np.float64)[..., None]


def decode(q, kc, vc, ks, vs, tables, lens, scale):
    """The definition of single-token attention over the cache, and the largest sums that its
    error bounds need: (out, sum_p w|v|, largest sum_d |q k| * |scale|, largest |v|)."""
    B, Hq, D = q.shape
    NB, bs, Hkv, _ = kc.shape
    G = Hq // Hkv
    out = np.zeros((B, Hq, D))
    wabs = np.zeros((B, Hq, D))
    mag = np.zeros((B, Hq, 1))
    vmax = np.zeros((B, Hq, 1))
    for s in range(B):
        n = int(lens[s])
        if n == 0:
            continue
        ids = tables[s, : -(-n // bs)].astype(np.int64)
        k = values(kc[ids].reshape(-1, Hkv, D // 2), ks[ids].transpose(0, 2, 1).reshape(-1, Hkv))[:n]
        v = values(vc[ids].reshape(-1, Hkv, D // 2), vs[ids].transpose(0, 2, 1).reshape(-1, Hkv))[:n]
        for h in range(Hq):
            kh, vh = k[:, h // G], v[:, h // G]
            z = kh @ q[s, h] * scale
            w = np.exp(z - z.max())
            w /= w.sum()
            out[s, h] = w @ vh
            wabs[s, h] = w @ np.abs(vh)
            mag[s, h] = (np.abs(kh) @ np.abs(q[s, h])).max() * abs(scale)
            vmax[s, h] = np.abs(vh).max()
    return out, wabs, mag, vmax


def decode_tolerance(dtype, lens, D, out, wabs, mag, vmax):
    """What rounding allows an output to be off, element by element.

    - Output: half a step of its type, 2^-8 (bf16), 2^-11 (fp16) or 2^-24 relative.
    - Scores: D products summed in fp32 are off by at most D 2^-24 (2^-22 where the tensor
      core truncates) of sum |q k|; the exponent's argument is rounded once more.  A score
      off by e changes a normalised weight by at most a factor exp(2 e).
    - Weights: 16-bit types may round a weight to 8 bits for bf16 (two 4-bit terms: half a
      step of 2^-4 twice) and 11 for fp16, plus 2^-21 of a tile's largest weight: at most
      2^-14 of the largest value over 128 tokens, summed over tiles.
    - fp32 sums over L tokens and the exponential: (L + 64) 2^-23.
    - The smallest numbers: a weight below 2^-126 of the largest is below fp32's normal range
      and may count as zero (L 2^-126 of the largest value), and an output of fp16 is a
      multiple of 2^-24 (half a step: 2^-25), of the other types of 2^-133 or finer.
    """
    half_step = {"bf16": 2.0**-8, "f16": 2.0**-11, "f32": 2.0**-24}[dtype]
    weight = {"bf16": 2.0**-8, "f16": 2.0**-11 + 2.0**-12, "f32": 0.0}[dtype]
    floor = 0.0 if dtype == "f32" else 2.0**-14
    L = np.asarray(lens, np.float64)[:, None, None]
    score = (D + 8) * (2.0**-24 if dtype == "f32" else 2.0**-22) * mag
    rel = np.expm1(2 * score) + weight + (L + 64) * 2.0**-23
    least = (2.0**-25 if dtype == "f16" else 2.0**-134) + L * 2.0**-126 * vmax
    return half_step * np.abs(out) + rel * wabs + floor * vmax + least


def resize(tables, lens, target, ring, pool, rows, bs, num_blocks):
    """kv_resize_requests on Python lists and arrays, in place; returns (slots, query_start,
    error bits)."""
    B, MB = tables.shape
    R = len(ring)
    cap = MB * bs
    head, count = int(pool[0]), int(pool[1])
    err = 0
    if not (0 <= head < R and 0 <= count <= R):
        err, head, count = 32, 0, 0
    slots = np.full(rows, -1, np.int64)
    start = np.zeros(B + 1, np.int32)
    want = tokens = taken = 0
    returned = []
    for s in range(B):
        old, new = int(lens[s]), int(target[s])
        start[s] = min(tokens, 2**31 - 1)
        if not (0 <= old <= cap and 0 <= new <= cap):
            err |= 8
            continue
        had, has = -(-old // bs), -(-new // bs)
        if new <= old:
            returned += [int(tables[s, j]) for j in range(has, had)]
            lens[s] = new
            continue
        row0 = tokens
        tokens += new - old
        want += has - had
        if tokens > rows or (has > had and want > count):
            err |= 32
            continue
        for j in range(had, has):
            tables[s, j] = ring[(head + want - (has - had) + j - had) % R]
        if has > had:
            taken = want
        for i in range(new - old):
            p = old + i
            b = int(tables[s, p // bs])
            if 0 <= b < num_blocks:
                slots[row0 + i] = b * bs + p % bs
            else:
                err |= 1
        lens[s] = new
    start[B] = min(tokens, 2**31 - 1)
    for i, b in enumerate(returned):
        if count + i < R:
            ring[(head + count + i) % R] = b
    left = count + len(returned)
    if left > R:
        err |= 32
        left = R
    pool[0] = (head + taken) % R
    pool[1] = left - taken
    return slots, start, err
