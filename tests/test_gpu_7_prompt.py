"""Prompt operators on the GPU against 64-bit definitions: scaled rotary tables, query / key
norm with rotation, attention of packed prompts, projections with their epilogue, and one
encoder layer made of them whose rows feed the image model.

Tolerances (u = 2^-8, the half step of bf16; 2^-24 that of fp32) are bounds of the
arithmetic, element by element:

* rope table: the angle is pos * w in fp64 (w off by ~2 ulp, one rounding of the product:
  3 |pos| 2^-53 < |pos| 2^-51), the reduced angle is rounded to fp32 (2^-25), the fp32 sine
  and cosine are within 2 ulp (2^-23), the product with the magnitude rounds twice.
* norm and rotation: sum of squares 13 roundings, root and quotient 2, products 2, rotation
  3, all below 32 half steps of fp32 on values up to 2 max|x|: 2^-18 max|x| of the head,
  plus the store.
* attention: each P is rounded to bf16 (u), and the store rounds once (u).  With A = sum p |v|
  the error is at most (u (1 + u) + d) A + u |O|, d = what fp32 adds: the logits, products
  of head_dim terms accumulated at 2^-23 a step, move p by scale (head_dim + 2) 2^-23
  max_j sum |q k_j| relative, twice (numerator and sum); PV accumulates up to m keys and
  the sum m / 8 at 2^-23 a step.
* linear: K / 16 accumulator steps of 2^-23, each on a partial sum below ~4 times the random
  walk T = sqrt(sum (a w)^2), plus 16 for the steps inside; activations with slope <= 1.13
  and relative error (exp of y at 2^-22 |y|) 2^-20 (1 + |y|); the store.
"""
import numpy as np
import pytest
import torch

import stream_diffusion_transformer_s3_b200 as Z
from _gpu import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rnd(seed, *shape, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def store_u(dtype):
    return U if dtype == torch.bfloat16 else 2.0 ** -24


def check(got, ref, bound, label):
    assert Z.zdit_device_status() == 0
    got, ref = got.double(), ref.double()
    assert torch.isfinite(got).all(), f"{label}: non-finite values"
    worst = ((got - ref).abs() / bound.clamp_min(1e-300)).max().item() if got.numel() else 0.0
    print(f"{label}: worst element at {worst:.3f} of its bound")
    assert worst <= 1.0, f"{label}: {worst:.3f} of the bound"


# ------------------------------------------------------------------ rotary tables
def frequencies(d, theta, sc):
    i = np.arange(d // 2, dtype=np.longdouble)
    w = np.longdouble(theta) ** (-2 * i / d)
    if sc is None or sc.kind == Z.ROPE_SCALE_NONE:
        return w
    f = np.longdouble(sc.factor)
    if sc.kind == Z.ROPE_SCALE_LINEAR:
        return w / f
    if sc.kind == Z.ROPE_SCALE_NTK:
        return (np.longdouble(theta) * f ** (np.longdouble(d) / (d - 2))) ** (-2 * i / d)
    pi = np.longdouble("3.14159265358979323846264338327950288")
    turns = np.longdouble(sc.original_len) * w / (2 * pi)
    g = np.clip((turns - sc.beta_slow) / (np.longdouble(sc.beta_fast) - np.longdouble(sc.beta_slow)), 0, 1)
    return w * g + w / f * (1 - g)


@pytest.mark.parametrize("T,d,theta,sc,first", [
    (1, 2, 1e4, None, 0),
    (5, 4, 1e4, Z.RopeScaling(Z.ROPE_SCALE_NTK, 8.0), -3),
    (77, 128, 1e6, None, 0),
    (777, 96, 5e5, Z.RopeScaling(Z.ROPE_SCALE_LINEAR, 4.0), 1 << 20),
    (333, 128, 1e6, Z.RopeScaling(Z.ROPE_SCALE_YARN, 4.0, 32768.0, 32.0, 1.0, 1.1386), 100000),
    (64, 22, 1e4, Z.RopeScaling(Z.ROPE_SCALE_YARN, 2.0, 2048.0, 32.0, 1.0), 5),   # 11 pairs a row
    (9, 512, 1e4, Z.RopeScaling(Z.ROPE_SCALE_NTK, 2.0), 12345),
    (6, 128, 1e4, None, (1 << 31) - 6),                                            # the last positions
    (3000, 64, 1e4, Z.RopeScaling(), -1500),
])
def test_rope_table_scaled(T, d, theta, sc, first):
    pos = np.arange(first, first + T, dtype=np.int64)
    cs = torch.full((T + 1, d // 2), 7.0, device="cuda")
    sn = torch.full((T + 1, d // 2), 7.0, device="cuda")
    Z.zdit_rope_table_scaled(torch.tensor(pos.astype(np.int32), device="cuda"), d, theta, cs[:T], sn[:T], sc)
    assert Z.zdit_device_status() == 0
    ang = pos.astype(np.longdouble)[:, None] * frequencies(d, theta, sc)
    mag = 1.0 if sc is None else float(sc.magnitude)
    tol = mag * (2.0 ** -25 + 2.0 ** -23 + 2.0 ** -23 + np.abs(pos)[:, None] * 2.0 ** -51)
    for got, ref in ((cs, np.cos(ang)), (sn, np.sin(ang))):
        err = np.abs(got[:T].double().cpu().numpy() - (ref * mag).astype(np.float64))
        print(f"rope {T}x{d}: {np.max(err / tol):.3f} of the bound")
        assert (err <= tol).all()
        assert (got[T] == 7.0).all()


def test_rope_table_scaled_agrees_with_the_three_axis_table():
    pos = torch.arange(50, device="cuda", dtype=torch.int32)
    a = [torch.empty(50, 64, device="cuda") for _ in range(4)]
    Z.zdit_rope_table_scaled(pos, 128, 1e4, a[0], a[1])
    Z.zdit_rope_table(torch.stack([pos, pos, pos], 1).contiguous(), (128, 0, 0), 1e4, a[2], a[3])
    assert (a[0] - a[2]).abs().max() < 2.0 ** -22 and (a[1] - a[3]).abs().max() < 2.0 ** -22


# ------------------------------------------------------------------ query / key norm and rotation
def norm_rotate(x, w, cos, sin, layout, rot, eps):
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    scale = x.abs().amax(-1, keepdim=True)
    y = x.clone()
    if rot:
        c, s = cos.double()[:, None], sin.double()[:, None]
        ia = torch.arange(rot // 2, device="cuda")
        ia, ib = (2 * ia, 2 * ia + 1) if layout == Z.ROPE_INTERLEAVED else (ia, ia + rot // 2)
        y[..., ia] = x[..., ia] * c - x[..., ib] * s
        y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return y, scale


def tables(T, rot, seed=3):
    ang = torch.rand(T, rot // 2, generator=torch.Generator().manual_seed(seed)).double() * 100
    return ang.cos().float().cuda(), ang.sin().float().cuda()


@pytest.mark.parametrize("layout", [Z.ROPE_HALF, Z.ROPE_INTERLEAVED])
@pytest.mark.parametrize("T,nq,nk,hd,rot,src,dst,norm", [
    (1, 1, 0, 8, 8, "f", "b", True),
    (1, 32, 8, 128, 128, "b", "b", True),
    (133, 32, 8, 128, 128, "f", "b", True),
    (257, 5, 5, 128, 32, "b", "b", True),       # a quarter of the head
    (64, 7, 1, 64, 64, "b", "f", True),
    (33, 3, 2, 80, 40, "b", "b", True),         # head of 10 lanes, halves of 20 elements
    (50, 6, 2, 96, 96, "f", "f", True),
    (50, 6, 2, 96, 6, "b", "b", True),          # 3 pairs
    (19, 2, 1, 256, 128, "b", "b", True),
    (19, 2, 1, 256, 256, "f", "b", False),
    (40, 4, 4, 128, 0, "b", "b", True),         # norm only
    (40, 4, 4, 64, 64, "b", "b", False),        # rotation only
])
def test_qk_norm_rope(T, nq, nk, hd, rot, src, dst, norm, layout):
    ty = {"f": torch.float32, "b": torch.bfloat16}
    row = (nq + 2 * nk) * hd + 16  # q | k | v | something else
    qkv = rnd(T * hd + rot, T, row, scale=3.0, dtype=ty[src])
    q, k = qkv[:, :nq * hd].view(T, nq, hd), qkv[:, nq * hd:(nq + nk) * hd].view(T, nk, hd)
    wq = 1 + 0.3 * rnd(1, hd, dtype=torch.float32) if norm else None
    wk = 1 + 0.3 * rnd(2, hd, dtype=torch.float32) if norm else None
    cos, sin = tables(T, rot) if rot else (None, None)
    qo = torch.full((T + 1, nq, hd), 99.0, device="cuda", dtype=ty[dst])
    ko = torch.full((nk, T + 1, hd), 99.0, device="cuda", dtype=ty[dst])  # head-major, as a cache may be
    Z.zdit_qk_norm_rope(q, k if nk else None, qo[:T], ko.transpose(0, 1)[:T] if nk else None, wq, wk, cos, sin, rot,
                        layout, eps=1e-6)
    for got, x, w, n in ((qo[:T], q, wq, nq), (ko.transpose(0, 1)[:T], k, wk, nk)):
        if n == 0:
            continue
        ref, scale = norm_rotate(x, w, cos, sin, layout, rot, 1e-6)
        check(got, ref, store_u(ty[dst]) * ref.abs() + 2.0 ** -18 * scale, f"qk {T}x{n}x{hd}/{rot}")
    assert (qo[T] == 99).all() and (ko[:, T] == 99).all()


def test_qk_norm_rope_in_place_touches_only_its_heads():
    T, nq, nk, hd = 61, 8, 2, 128
    qkv = rnd(5, T, (nq + 2 * nk) * hd)
    before = qkv.clone()
    q, k = qkv[:, :nq * hd].view(T, nq, hd), qkv[:, nq * hd:(nq + nk) * hd].view(T, nk, hd)
    w = 1 + 0.3 * rnd(1, hd, dtype=torch.float32)
    cos, sin = tables(T, hd)
    apart = [torch.empty(T, n, hd, device="cuda", dtype=torch.bfloat16) for n in (nq, nk)]
    Z.zdit_qk_norm_rope(q, k, *apart, w, w, cos, sin, hd)
    Z.zdit_qk_norm_rope(q, k, q, k, w, w, cos, sin, hd)
    assert torch.equal(q, apart[0]) and torch.equal(k, apart[1])
    assert torch.equal(qkv[:, (nq + nk) * hd:], before[:, (nq + nk) * hd:])


def test_qk_norm_rope_zero_and_large_rows():
    # a head of zeros stays zero (eps), one near the largest bf16 does not overflow its sum
    T, hd = 4, 128
    q = torch.zeros(T, 1, hd, device="cuda", dtype=torch.bfloat16)
    q[1] = 1e18
    q[2] = 3e-20
    q[3, 0, ::2] = -5.0
    cos, sin = tables(T, hd)
    out = torch.empty_like(q)
    Z.zdit_qk_norm_rope(q, None, out, None, torch.ones(hd, device="cuda"), None, cos, sin, hd)
    ref, scale = norm_rotate(q, torch.ones(hd, device="cuda"), cos, sin, Z.ROPE_HALF, hd, 1e-6)
    check(out, ref, U * ref.abs() + 2.0 ** -18 * scale, "qk extremes")
    assert (out[0] == 0).all()


# ------------------------------------------------------------------ attention
def attention_ref(q, k, v, q_len, kv_len, kv_start, causal, scale):
    """(O, bound) of the definition in 64 bits, per sequence and head."""
    H, Hkv, hd = q.shape[1], k.shape[1], q.shape[2]
    O = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    B = torch.zeros_like(O)
    t0 = 0
    for n, m, s0 in zip(q_len, kv_len, kv_start):
        if n and m:
            ks, vs = k[s0:s0 + m].double(), v[s0:s0 + m].double()
            for h in range(H):
                qh, kh, vh = q[t0:t0 + n, h].double(), ks[:, h * Hkv // H], vs[:, h * Hkv // H]
                x = qh @ kh.T * scale
                ok = torch.ones(n, m, dtype=torch.bool, device="cuda")
                if causal:
                    ok = ok.tril(m - n)
                x = x.masked_fill(~ok, -torch.inf)
                p = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-1e300)).masked_fill(~ok, 0.0)
                den = p.sum(-1, keepdim=True)
                p = torch.where(den > 0, p / den.clamp_min(1e-300), torch.zeros_like(p))
                O[t0:t0 + n, h] = p @ vh
                A = p @ vh.abs()
                dl = scale * (hd + 2) * 2.0 ** -23 * (qh.abs() @ kh.abs().T).amax(-1, keepdim=True)
                d = 2 * dl + (2 * m + 64) * 2.0 ** -23
                B[t0:t0 + n, h] = (U * (1 + U) + d) * A + U * O[t0:t0 + n, h].abs()
        t0 += n
    return O, B


def workspace(batch, H, Hkv, hd, causal=True):
    """What the call needs, every byte set so that a value read before it is written is NaN."""
    need = Z.prompt_attention_workspace_bytes(batch, H, Hkv, hd, causal)
    return torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None


def run_attention(q_len, kv_len=None, kv_start=None, H=8, Hkv=2, hd=128, causal=True, seed=0, scale=0.0, gap=0,
                  qscale=1.0, head_major=False, label=""):
    """One call on inputs with NaN in every row of k and v that no sequence owns and a
    sentinel in the rows of o behind the last sequence; returns o."""
    lens = q_len if kv_len is None else kv_len
    starts = kv_start if kv_start is not None else [sum(lens[:b]) for b in range(len(lens))]
    T, R = sum(q_len), max([s + m for s, m in zip(starts, lens)] + [0]) + gap
    q = rnd(seed + 1, T + 2, H, hd, scale=qscale)
    k, v = rnd(seed + 2, R, Hkv, hd), rnd(seed + 3, R, Hkv, hd)
    owned = torch.zeros(R, dtype=torch.bool)
    for s, m in zip(starts, lens):
        owned[s:s + m] = True
    k[~owned.cuda()] = torch.nan
    v[~owned.cuda()] = torch.nan
    if head_major:
        k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v))
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    q[T:] = torch.nan
    o = torch.full((T + 3, H, hd), 17.0, device="cuda", dtype=torch.bfloat16)
    if head_major:
        o = o.transpose(0, 1).contiguous().transpose(0, 1)
    batch = Z.PromptBatch(q_len, kv_len, kv_start)
    ws = workspace(batch, H, Hkv, hd, causal)
    Z.zdit_prompt_attention(q, k, v, o, batch, ws, causal=causal, scale=scale)
    sc = scale if scale else hd ** -0.5
    ref, bound = attention_ref(q[:T], k, v, q_len, lens, starts, causal, sc)
    check(o[:T], ref, bound, label or f"attention q {q_len} kv {lens} {H}/{Hkv}x{hd} split {ws is not None}")
    assert (o[T:] == 17.0).all()
    return o, (q, k, v, batch, ws)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q_len,H,Hkv", [
    ((1,), 1, 1),
    ((1, 2, 3), 4, 1),
    ((127, 128, 129), 2, 2),               # a tile less one, a tile, a tile and one
    ((255, 1, 257), 3, 3),                 # pairs of tiles
    ((31, 32, 33, 64, 65), 8, 2),          # groups of 4: tiles of 32 tokens
    ((40, 43), 6, 2),                      # groups of 3: 42 tokens and 2 unused rows
    ((10, 300), 14, 2),                    # groups of 7
    ((50,), 64, 1),                        # 64 heads on one key head: 2 tokens a tile
    ((0, 5, 0, 9), 4, 4),                  # empty sequences
    ((1000, 7), 4, 2),
])
def test_prompt_attention_whole_prompts(q_len, H, Hkv, hd):
    run_attention(q_len, H=H, Hkv=Hkv, hd=hd, gap=3, seed=sum(q_len))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q_len,kv_len,kv_start", [
    ((1, 1, 1), (1, 128, 129), None),                       # single tokens
    ((1, 1), (5000, 4097), (0, 6000)),                      # split keys, slots with a gap
    ((3, 17), (900, 2000), (5, 905)),
    ((37, 37, 37), (1500, 1500, 1500), (0, 0, 0)),          # the same prefix three times
    ((200, 1), (1000, 3000), (3000, 0)),                    # slots in another order
    ((5, 4, 3), (0, 2, 3), (0, 0, 2)),                      # no keys; fewer keys than rows
    ((300,), (130,), (0,)),                                 # first rows see nothing
    ((2,), (9001,), (77,)),
])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_attention_prefixes_and_single_tokens(q_len, kv_len, kv_start, hd, causal):
    run_attention(q_len, kv_len, kv_start, H=8, Hkv=2, hd=hd, causal=causal, gap=200, seed=sum(kv_len))


def test_prompt_attention_rows_without_keys_are_zero():
    o, _ = run_attention((300,), (130,), (0,), H=4, Hkv=2)
    assert (o[:170] == 0).all() and (o[170:300] != 0).any()
    o, _ = run_attention((5,), (0,), (0,), H=4, Hkv=2)
    assert (o[:5] == 0).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q_len,kv_len", [((150,), (150,)), ((100, 40), (130, 700)), ((3, 90), (2000, 90))])
def test_prompt_attention_nonfinite_rows_reach_only_rows_that_see_them(q_len, kv_len, hd):
    H, Hkv = 8, 2
    starts = [sum(kv_len[:b]) for b in range(len(kv_len))]
    q, k, v = rnd(1, sum(q_len), H, hd), rnd(2, sum(kv_len), Hkv, hd), rnd(3, sum(kv_len), Hkv, hd)
    batch = Z.PromptBatch(q_len, kv_len)
    ws = workspace(batch, H, Hkv, hd)
    clean, o = torch.empty_like(q), torch.empty_like(q)
    Z.zdit_prompt_attention(q, k, v, clean, batch, ws)
    bad = [(0, kv_len[0] - 1, torch.nan, 3), (0, kv_len[0] - 3, torch.inf, hd - 1),
           (len(kv_len) - 1, kv_len[-1] - q_len[-1] // 2, -torch.inf, 17)]
    want = clean.double()
    for b, j, x, d in bad:
        v[starts[b] + j, 0, d] = x                       # key head 0: query heads 0..3
        first = j - (kv_len[b] - q_len[b])               # first row of the sequence that sees it
        rows = slice(sum(q_len[:b]) + max(first, 0), sum(q_len[:b + 1]))
        want[rows, :H // Hkv, d] += x
    Z.zdit_prompt_attention(q, k, v, o, batch, ws)
    assert Z.zdit_device_status() == 0
    assert torch.equal(o.isnan(), want.isnan()) and torch.equal(o.isinf(), want.isinf())
    assert torch.equal(o[want.isinf()].double(), want[want.isinf()])
    # what was finite is as before (a cleaned tile sums the same finite values)
    assert torch.equal(o[want.isfinite()], clean[want.isfinite()])
    # an infinite or NaN key changes the rows that see it and no others
    k[starts[-1] + kv_len[-1] - 1, 1] = torch.nan
    Z.zdit_prompt_attention(q, k, v, o, batch, ws)
    assert o[-1, H // Hkv:].isnan().all()
    assert torch.equal(o[:-1, H // Hkv:], clean[:-1, H // Hkv:])


@pytest.mark.parametrize("hd", [64, 128])
def test_prompt_attention_uneven_strides(hd):
    # rows with something between and after the heads, strides that do not divide one another
    H, Hkv, n = 6, 3, 77
    buf = rnd(5, n, (H + 2 * Hkv) * (hd + 8) + 24)
    cut = lambda first, heads: buf[:, first * (hd + 8):(first + heads) * (hd + 8)].view(n, heads, hd + 8)[..., :hd]
    q, k, v = cut(0, H), cut(H, Hkv), cut(H + Hkv, Hkv)
    o = torch.full((n, H, hd + 16), 5.0, device="cuda", dtype=torch.bfloat16)
    batch = Z.PromptBatch([n])
    Z.zdit_prompt_attention(q, k, v, o[..., :hd], batch, workspace(batch, H, Hkv, hd))
    ref, bound = attention_ref(q, k, v, [n], [n], [0], True, hd ** -0.5)
    check(o[..., :hd], ref, bound, "uneven strides")
    assert (o[..., hd:] == 5.0).all()


@pytest.mark.parametrize("hd", [64, 128])
def test_prompt_attention_head_major_buffers(hd):
    run_attention((70, 133), H=6, Hkv=3, hd=hd, head_major=True)
    run_attention((1, 1), (700, 3000), (0, 700), H=6, Hkv=3, hd=hd, head_major=True)


def test_prompt_attention_scale_and_peaked_rows():
    run_attention((200,), H=4, Hkv=1, scale=0.5)
    run_attention((64, 300), H=4, Hkv=2, qscale=8.0)       # a row's weight on few keys
    run_attention((1,), (6000,), (0,), H=8, Hkv=1, qscale=8.0)


def test_prompt_attention_reference_maximum_moves():
    # logits that grow along the keys by far more than the rescale threshold, and shrink
    for sign in (1.0, -1.0):
        n, H, hd = 700, 2, 128
        q = torch.full((n, H, hd), 0.5, device="cuda", dtype=torch.bfloat16)
        ramp = sign * torch.linspace(0, 6, n, device="cuda")[:, None, None]
        k = (rnd(3, n, H, hd, dtype=torch.float32) * 0.1 + ramp).bfloat16()
        v = rnd(4, n, H, hd)
        for rows in (n, 1):
            o = torch.empty(rows, H, hd, device="cuda", dtype=torch.bfloat16)
            b = Z.PromptBatch([rows], [n])
            Z.zdit_prompt_attention(q[:rows], k, v, o, b, workspace(b, H, H, hd))
            ref, bound = attention_ref(q[:rows], k, v, [rows], [n], [0], True, hd ** -0.5)
            check(o, ref, bound, f"moving maximum {sign} {rows}")


def test_prompt_attention_long_prompt():
    run_attention((4500, 700), H=4, Hkv=1, seed=9)


def test_prompt_attention_equals_joint_attention_without_mask():
    lengths, H = (130, 333), 3
    T = sum(lengths)
    q, k, v = (rnd(i, T, H, 128) for i in (1, 2, 3))
    a, b = torch.empty_like(q), torch.empty_like(q)
    batch = Z.PromptBatch(lengths)
    Z.zdit_prompt_attention(q, k, v, a, batch, workspace(batch, H, H, 128, False), causal=False)
    Z.zdit_joint_attention(q.view(T, -1), k.view(T, -1), v.view(T, -1), b.view(T, -1), Z.DeviceVarlen([0, 130, T]), H)
    ref, bound = attention_ref(q, k, v, lengths, lengths, (0, 130), False, 128 ** -0.5)
    check(a, ref, bound, "unmasked")
    check(b, ref, bound, "joint attention")


def test_prompt_attention_is_deterministic_and_replays():
    # a split call: the same bits every time, eager, on another stream and from a graph
    o, (q, k, v, batch, ws) = run_attention((1, 2, 1), (5000, 777, 3000), (0, 5000, 6000), H=8, Hkv=2)
    first = o[:4].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2 = torch.zeros_like(o)
        Z.zdit_prompt_attention(q, k, v, o2, batch, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o2[:4], first)
    o3 = torch.zeros_like(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Z.zdit_prompt_attention(q, k, v, o3, batch, ws)
    for _ in range(3):
        o3.zero_()
        g.replay()
        assert torch.equal(o3[:4], first)
    # replayed on new data in the same buffers
    q.mul_(0.5)
    g.replay()
    ref, bound = attention_ref(q[:4], k, v, [1, 2, 1], [5000, 777, 3000], [0, 5000, 6000], True, 128 ** -0.5)
    check(o3[:4], ref, bound, "replay on new data")


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q_len,kv_len", [
    ((1,) * 8, (8191, 2501, 6000, 3333, 4097, 5555, 7001, 2999)),
    (tuple(range(30, 400, 17)), None),
    ((333, 500, 1), (4001, 2999, 8001)),
])
def test_prompt_attention_under_load_back_to_back(q_len, kv_len, hd):
    # enough work to keep every SM and the memory busy, so that the warps of a CTA drift apart;
    # sequences that end inside a key tile; calls queued behind one another on two sets of buffers
    H, Hkv = 32, 8
    lens = q_len if kv_len is None else kv_len
    cap = (max(lens) + 63) // 64 * 64
    starts = [b * cap for b in range(len(lens))] if kv_len else [sum(lens[:b]) for b in range(len(lens))]
    rows = starts[-1] + (cap if kv_len else lens[-1])
    batch = Z.PromptBatch(q_len, kv_len, starts)
    sets = []
    for i in range(2):
        q, k, v = rnd(10 + i, sum(q_len), H, hd), rnd(20 + i, rows, Hkv, hd), rnd(30 + i, rows, Hkv, hd)
        sets.append((q, k, v, workspace(batch, H, Hkv, hd)))
    torch.cuda.synchronize()
    outs = [[torch.empty_like(sets[i][0]) for _ in range(6)] for i in range(2)]
    for r in range(6):
        for i, (q, k, v, ws) in enumerate(sets):
            Z.zdit_prompt_attention(q, k, v, outs[i][r], batch, ws)
    for i, (q, k, v, ws) in enumerate(sets):
        ref, bound = attention_ref(q, k, v, q_len, lens, starts, True, hd ** -0.5)
        for r in range(6):
            check(outs[i][r], ref, bound, f"set {i} call {r}")
            assert torch.equal(outs[i][r], outs[i][0])


def test_prompt_attention_far_row_offsets():
    # key rows whose offsets pass 2^31 elements: 33 M rows of one head, the last ones used
    rows, hd = (1 << 25) + 1000, 64
    k = torch.empty(rows, 1, hd, device="cuda", dtype=torch.bfloat16)
    v = torch.empty(rows, 1, hd, device="cuda", dtype=torch.bfloat16)
    start = rows - 900
    k[start:], v[start:] = rnd(1, 900, 1, hd), rnd(2, 900, 1, hd)
    q = rnd(3, 40, 2, hd)
    o = torch.empty_like(q)
    b = Z.PromptBatch([40], [900], [start])
    Z.zdit_prompt_attention(q, k, v, o, b, workspace(b, 2, 1, hd))
    ref, bound = attention_ref(q, k[start:], v[start:], [40], [900], [0], True, hd ** -0.5)
    check(o, ref, bound, "far rows")


# ------------------------------------------------------------------ linear
def linear_ref(a, w, bias, act, residual, exact_product=False):
    A, W = a.double(), w.double()
    y = A @ W.T
    T = (A.square() @ W.square().T).sqrt()
    K = a.shape[1]
    e = (0.0 if exact_product else 4 * (K / 16 + 16) * 2.0 ** -23) * T
    if bias is not None:
        y = y + bias.double()
        e = e + 2.0 ** -23 * y.abs()
    f = y
    if act == Z.ACT_SILU:
        f = y * torch.sigmoid(y)
    elif act == Z.ACT_GELU:
        f = 0.5 * y * torch.special.erfc(-y / 2 ** 0.5)
    elif act == Z.ACT_GELU_TANH:
        f = y * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (y + 0.044715 * y ** 3))
    if act != Z.ACT_NONE:
        # relative error of the exponential: its argument (y, or up to ~1.6 y (1 + y^2 / 22)
        # for the tanh form) in fp32, and 2^-22 of the function itself
        arg = y.abs() * (1 + (0.1 * y.square() if act == Z.ACT_GELU_TANH else y.abs() if act == Z.ACT_GELU else 0))
        e = 1.13 * e + 2.0 ** -20 * (1 + arg) * f.abs()
    if residual is not None:
        f = f + residual.double()
        e = e + 2.0 ** -23 * (f.abs() + residual.double().abs())
    return f, e


SHAPES = [
    (1, 1, 1), (1, 1, 8), (3, 5, 7), (1, 2560, 4096), (5, 2560, 4096), (16, 129, 64), (17, 256, 65), (33, 300, 1000),
    (64, 1024, 2560), (65, 2560, 320), (133, 9728, 256), (128, 128, 128), (200, 777, 2560), (257, 255, 250),
    (600, 1111, 2563), (1000, 512, 64), (2049, 640, 3840),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act,bias,res,out", [
    (Z.ACT_NONE, False, None, "f"),
    (Z.ACT_SILU, True, None, "b"),
    (Z.ACT_GELU, True, "f", "b"),
    (Z.ACT_GELU_TANH, False, "b", "f"),
])
def test_linear(M, N, K, act, bias, res, out):
    ty = {"f": torch.float32, "b": torch.bfloat16}
    Kp = (K + 7) // 8 * 8 + 8
    a, w = rnd(1, M, Kp), rnd(2, N, Kp, scale=K ** -0.5)
    a[:, K:], w[:, K:] = torch.nan, torch.nan  # columns past K are never used
    a, w = a[:, :K], w[:, :K]
    b = rnd(3, N, dtype=torch.float32) if bias else None
    r = rnd(4, M, N + 3, scale=2.0, dtype=ty[res])[:, :N] if res else None
    o = torch.full((M + 1, N + 5), 9.0, device="cuda", dtype=ty[out])
    Z.zdit_linear(a, w, o[:M, :N], bias=b, act=act, residual=r)
    ref, e = linear_ref(a, w, b, act, r)
    check(o[:M, :N], ref, e + store_u(ty[out]) * ref.abs(), f"linear {M}x{N}x{K} act {act}")
    assert (o[M] == 9).all() and (o[:, N:] == 9).all()


@pytest.mark.parametrize("M,N,K", [(5, 2560, 512), (133, 520, 2560), (700, 768, 1024)])
@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
def test_linear_residual_in_place(M, N, K, ty):
    a, w, x = rnd(1, M, K), rnd(2, N, K, scale=K ** -0.5), rnd(3, M, N, dtype=ty)
    ref, e = linear_ref(a, w, None, Z.ACT_NONE, x)
    Z.zdit_linear(a, w, x, residual=x)
    check(x, ref, e + store_u(ty) * ref.abs(), "residual in place")


@pytest.mark.parametrize("act", [Z.ACT_SILU, Z.ACT_GELU, Z.ACT_GELU_TANH])
def test_linear_activation_tails(act):
    # values from -60 to 60 through an identity product
    n = 64
    y = torch.linspace(-60, 60, n, device="cuda").bfloat16()
    a = y[:, None] * torch.eye(n, device="cuda", dtype=torch.bfloat16)
    o = torch.empty(n, n, device="cuda")
    Z.zdit_linear(a, torch.eye(n, device="cuda", dtype=torch.bfloat16), o, act=act)
    ref, e = linear_ref(a, torch.eye(n, device="cuda", dtype=torch.bfloat16), None, act, None, exact_product=True)
    # products are exact here: only the activation's own error counts, and fp32's smallest values
    check(o, ref, e + 2.0 ** -24 * ref.abs() + 2.0 ** -126, "tails")


def test_linear_is_deterministic_and_replays():
    a, w = rnd(1, 5, 4096), rnd(2, 2560, 4096, scale=1 / 64)
    x = rnd(3, 5, 2560, dtype=torch.float32)
    o = [torch.empty_like(x) for _ in range(2)]
    Z.zdit_linear(a, w, o[0], residual=x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Z.zdit_linear(a, w, o[1], residual=x)
    for _ in range(3):
        o[1].zero_()
        g.replay()
        assert torch.equal(o[0], o[1])


# ------------------------------------------------------------------ together
class Layer:
    """Attention half of a causal prompt layer, in 64 bits with the library's roundings left
    out, and through the library."""

    def __init__(self, D, H, Hkv, hd):
        self.D, self.H, self.Hkv, self.hd = D, H, Hkv, hd
        self.w_qkv = rnd(11, (H + 2 * Hkv) * hd, D, scale=D ** -0.5)
        self.w_o = rnd(12, D, H * hd, scale=(H * hd) ** -0.5)
        self.nq, self.nk = (1 + 0.2 * rnd(s, hd, dtype=torch.float32) for s in (13, 14))

    def exact(self, x, pos, q_len):
        H, Hkv, hd = self.H, self.Hkv, self.hd
        T = x.shape[0]
        qkv = x.double() @ self.w_qkv.double().T
        q, k, v = (qkv[:, a:b].reshape(T, -1, hd) for a, b in ((0, H * hd), (H * hd, (H + Hkv) * hd),
                                                               ((H + Hkv) * hd, (H + 2 * Hkv) * hd)))
        ang = pos.double()[:, None] * 1e6 ** (-torch.arange(hd // 2, device="cuda", dtype=torch.float64) * 2 / hd)
        q, _ = norm_rotate(q, self.nq, ang.cos(), ang.sin(), Z.ROPE_HALF, hd, 1e-6)
        k, _ = norm_rotate(k, self.nk, ang.cos(), ang.sin(), Z.ROPE_HALF, hd, 1e-6)
        starts = [sum(q_len[:b]) for b in range(len(q_len))]
        o, _ = attention_ref(q, k, v, q_len, q_len, starts, True, hd ** -0.5)
        return x.double() + o.reshape(T, -1) @ self.w_o.double().T

    def run(self, x, x16, pos, q_len, out, buf):
        H, Hkv, hd = self.H, self.Hkv, self.hd
        T = x.shape[0]
        qkv, cos, sin, o, ws = buf
        Z.zdit_rope_table_scaled(pos, hd, 1e6, cos, sin)
        Z.zdit_linear(x16, self.w_qkv, qkv)
        q, k, v = (qkv[:, a:b].view(T, -1, hd) for a, b in ((0, H * hd), (H * hd, (H + Hkv) * hd),
                                                            ((H + Hkv) * hd, (H + 2 * Hkv) * hd)))
        Z.zdit_qk_norm_rope(q, k, q, k, self.nq, self.nk, cos, sin, hd, Z.ROPE_HALF)
        batch = Z.PromptBatch(q_len)
        Z.zdit_prompt_attention(q, k, v, o, batch, ws)
        Z.zdit_linear(o.view(T, -1), self.w_o, out, residual=x)


@pytest.mark.parametrize("q_len", [(45, 1), (300, 7, 41)])
def test_prompt_layer_feeds_the_image_model(q_len):
    L = Layer(128, 4, 2, 64)
    T = sum(q_len)
    x16 = rnd(20, T, L.D)
    x = x16.float()
    pos = torch.cat([torch.arange(n) for n in q_len]).to(device="cuda", dtype=torch.int32)
    out = torch.empty_like(x)
    buf = (torch.empty(T, 8 * 64, device="cuda", dtype=torch.bfloat16), torch.empty(T, 32, device="cuda"),
           torch.empty(T, 32, device="cuda"), torch.empty(T, 4, 64, device="cuda", dtype=torch.bfloat16),
           workspace(Z.PromptBatch(q_len), 4, 2, 64))
    L.run(x, x16, pos, q_len, out, buf)
    assert Z.zdit_device_status() == 0
    ref = L.exact(x, pos, q_len)
    # the update carries 4 bf16 roundings (projected row, rotated head, P, attention row): u sqrt(4 / 3)
    # of its scale on average; 4 u bounds the ratio of the norms
    err = (out.double() - ref).norm() / (ref - x.double()).norm()
    print(f"layer update rel {err:.2e}")
    assert err < 4 * U
    # the same run from a graph gives the same bits
    again = torch.zeros_like(out)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        L.run(x, x16, pos, q_len, again, buf)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.run(x, x16, pos, q_len, again, buf)
    again.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    if len(q_len) == 2:
        # the rows are caption features of the image model
        from stream_diffusion_transformer_s3_b200 import synth
        d = synth.BlockDims(dim=256, n_heads=2, head_dim=128, ffn_hidden=384)
        W = synth.stack_weights(0, d, n_noise=1, n_context=1, n_main=1, cap_dim=128)
        case = synth.stack_case(0, 8, 8, [64, 32], list(q_len), [0.5, 0.5], cap_dim=128)
        import oracle as O
        case["caps"] = out.cpu().numpy()
        dims = Z.Dims(dim=256, n_heads=2, ffn_hidden=384)
        stack = Z.DeviceStack(W, dims, 1, 1, 1, patch_dim=64, cap_dim=128)
        patches = torch.as_tensor(np.ascontiguousarray(case["patches"]), dtype=torch.float32).cuda()
        call = Z.StackCall(case["grid"], case["n_caps"], case["n_valids"], case["t"], patches, out)
        ws = torch.empty(Z.stack_workspace_bytes(stack, call), dtype=torch.uint8, device="cuda")
        vel = torch.empty(2, 64, 64, device="cuda")
        Z.zdit_stack_forward(stack, call, vel, ws)
        assert Z.zdit_device_status() == 0
        want = O.stack_forward(case, W, d)
        got = vel.double().cpu().numpy()
        assert np.linalg.norm(got - want) / np.linalg.norm(want) <= 2e-2


def test_prompt_rows_of_a_later_call_match_the_whole_prompt():
    # the prompt in one call, or as a kept prefix, a middle and single tokens over the cache
    H, Hkv, hd, n = 8, 2, 128, 400
    q, k, v = rnd(1, n, H, hd), rnd(2, n, Hkv, hd), rnd(3, n, Hkv, hd)
    whole = torch.empty_like(q)
    b = Z.PromptBatch([n])
    Z.zdit_prompt_attention(q, k, v, whole, b, workspace(b, H, Hkv, hd))
    parts = torch.empty_like(q)
    at = 0
    for m in (250, 147, 1, 1, 1):
        b = Z.PromptBatch([m], [at + m])
        Z.zdit_prompt_attention(q[at:at + m], k, v, parts[at:at + m], b, workspace(b, H, Hkv, hd))
        at += m
    ref, bound = attention_ref(q, k, v, [n], [n], [0], True, hd ** -0.5)
    check(whole, ref, bound, "whole")
    check(parts, ref, bound, "in parts")


def test_prompt_layers_on_two_streams_at_once():
    # eager calls and captured graphs of two streams, each with buffers of its own
    L = Layer(128, 4, 2, 64)
    runs = []
    for i, q_len in enumerate([(300, 7, 41), (1, 900)]):
        T = sum(q_len)
        x16 = rnd(30 + i, T, L.D)
        pos = torch.cat([torch.arange(n) for n in q_len]).to(device="cuda", dtype=torch.int32)
        buf = (torch.empty(T, 8 * 64, device="cuda", dtype=torch.bfloat16), torch.empty(T, 32, device="cuda"),
               torch.empty(T, 32, device="cuda"), torch.empty(T, 4, 64, device="cuda", dtype=torch.bfloat16),
               workspace(Z.PromptBatch(q_len), 4, 2, 64))
        x = x16.float()
        alone = torch.empty_like(x)
        L.run(x, x16, pos, q_len, alone, buf)
        runs.append((torch.cuda.Stream(), x, x16, pos, q_len, buf, alone, [torch.zeros_like(x) for _ in range(8)]))
    torch.cuda.synchronize()
    for r in range(8):
        for s, x, x16, pos, q_len, buf, alone, outs in runs:
            with torch.cuda.stream(s):
                L.run(x, x16, pos, q_len, outs[r], buf)
    torch.cuda.synchronize()
    for *_, alone, outs in runs:
        assert all(torch.equal(o, alone) for o in outs)
    graphs = []
    for s, x, x16, pos, q_len, buf, alone, outs in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            L.run(x, x16, pos, q_len, outs[0], buf)
        outs[0].zero_()
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(8):
        for g, (s, *_) in zip(graphs, runs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for *_, alone, outs in runs:
        assert torch.equal(outs[0], alone)
    assert Z.zdit_device_status() == 0


@pytest.mark.parametrize("hd", [64, 128])
def test_prompt_attention_many_sequences_on_the_same_keys(hd):
    # the largest batch; every other sequence continues the same prefix, the rest have their own keys
    H, Hkv = 4, 2
    q_len = [1 + b % 5 for b in range(128)]
    kv_len = [200 + b % 5 if b % 2 == 0 else 1 + 3 * b for b in range(128)]
    starts = [0 if b % 2 == 0 else 10 * b for b in range(128)]
    q = rnd(1, sum(q_len), H, hd)
    rows = max(s + n for s, n in zip(starts, kv_len))
    k, v = rnd(2, rows, Hkv, hd), rnd(3, rows, Hkv, hd)
    o = torch.empty_like(q)
    b = Z.PromptBatch(q_len, kv_len, starts)
    Z.zdit_prompt_attention(q, k, v, o, b, workspace(b, H, Hkv, hd))
    ref, bound = attention_ref(q, k, v, q_len, kv_len, starts, True, hd ** -0.5)
    check(o, ref, bound, "128 sequences")


def test_prompt_attention_without_query_rows_writes_nothing():
    q = rnd(1, 3, 2, 64)
    k = rnd(2, 9, 2, 64)
    o = torch.full_like(q, 5.0)
    Z.zdit_prompt_attention(q, k, k.clone(), o, Z.PromptBatch([0, 0], [4, 5]))
    torch.cuda.synchronize()
    assert (o == 5).all() and Z.zdit_device_status() == 0


# ------------------------------------------------------------------ rotations past a head's first chunks
@pytest.mark.parametrize("T", [1, 37])
@pytest.mark.parametrize("src,dst", [("b", "b"), ("f", "f")])
@pytest.mark.parametrize("hd,rot", [(24, 24), (40, 40), (72, 72), (80, 48), (80, 80), (88, 88), (96, 64), (104, 104),
                                    (112, 72), (192, 128), (200, 200), (248, 136)])
def test_qk_norm_rope_halves_past_the_first_chunks(hd, rot, T, src, dst):
    # heads that leave lanes of their group without elements, partners on both sides of the
    # element where the lanes' second chunks begin
    test_qk_norm_rope(T, 3, 2, hd, rot, src, dst, True, Z.ROPE_HALF)


# ------------------------------------------------------------------ host threads
@pytest.mark.parametrize("op", ["rope", "qk", "attention", "linear", "linear many rows", "gemm", "joint attention"])
def test_first_call_of_a_host_thread(op):
    # a thread on which nothing has touched the device yet: no torch call, no cudaSetDevice
    from threading import Thread
    T, H, hd = 40, 2, 128
    q, k, v = (rnd(i, T, H, hd) for i in (1, 2, 3))
    cos, sin = tables(T, hd)
    M = 4096 if op == "linear many rows" else 3
    a, w = rnd(5, M, 256), rnd(6, 4096, 256)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    out = {"rope": (T, hd // 2), "linear": (M, 4096), "linear many rows": (M, 4096), "gemm": (M, 4096)}.get(op, (T, H, hd))
    ty = torch.float32 if len(out) == 2 else torch.bfloat16
    o, want = (torch.zeros(out, device="cuda", dtype=ty) for _ in range(2))
    o2, batch, one = torch.zeros_like(o), Z.PromptBatch([T]), Z.DeviceVarlen([0, T])
    stream = torch.cuda.current_stream()
    calls = {
        "rope": lambda o: Z.zdit_rope_table_scaled(pos, hd, 1e4, o, o2, stream=stream),
        "qk": lambda o: Z.zdit_qk_norm_rope(q, None, o, None, None, None, cos, sin, hd, stream=stream),
        "attention": lambda o: Z.zdit_prompt_attention(q, k, v, o, batch, causal=False, stream=stream),
        "linear": lambda o: Z.zdit_linear(a, w, o, stream=stream),
        "linear many rows": lambda o: Z.zdit_linear(a, w, o, stream=stream),
        "gemm": lambda o: Z.zdit_gemm_bf16(a, w, o, stream=stream),
        "joint attention": lambda o: Z.zdit_joint_attention(*(x.view(T, -1) for x in (q, k, v, o)), one, H,
                                                            stream=stream),
    }
    assert Z.prompt_attention_workspace_bytes(batch, H, H, hd, False) == 0
    calls[op](want)
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            calls[op](o)
        except Exception as e:
            failed.append(e)

    t = Thread(target=work)
    t.start()
    t.join()
    assert not failed
    assert Z.zdit_device_status() == 0
    assert torch.equal(o, want)


def test_linear_from_host_threads_at_once():
    # calls whose tiles need different amounts of shared memory, queued by several threads at
    # once through the C call itself, so that they meet inside the library
    import ctypes as C
    from concurrent.futures import ThreadPoolExecutor
    from threading import Barrier
    N, K, rows = 256, 512, (1, 64, 144, 96) * 2
    start, call = Barrier(len(rows), timeout=60), Z.lib().zdit_linear
    w = rnd(2, N, K, scale=K ** -0.5)
    a = [rnd(3 + M, M, K) for M in rows]
    want, got = ([torch.zeros(M, N, device="cuda") for M in rows] for _ in range(2))
    for x, o in zip(a, want):
        Z.zdit_linear(x, w, o)
    torch.cuda.synchronize()

    def work(i):
        stream = torch.cuda.Stream()
        g = Z.LinearArgs(M=rows[i], N=N, K=K, a=a[i].data_ptr(), lda=K, w=w.data_ptr(), ldw=K, out=got[i].data_ptr(),
                         ld_out=N, out_dtype=1)
        start.wait()
        failed = sum(call(C.byref(g), stream.cuda_stream) != 0 for _ in range(5000))
        stream.synchronize()
        return failed

    with ThreadPoolExecutor(len(rows)) as pool:
        failed = list(pool.map(work, range(len(rows))))
    assert failed == [0] * len(rows)
    assert Z.zdit_device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))


# ------------------------------------------------------------------ errors of the host
@pytest.mark.parametrize("op", ["rope", "qk", "attention", "split attention", "linear", "linear many rows"])
def test_a_refused_launch_does_not_fail_the_next_call(op):
    # a launch on the default stream while a stream that waits for it is being captured is refused
    # by the runtime, on the host; the capture is given up, another call and the same one are made
    import ctypes as C
    rt = C.CDLL("libcudart.so.12")
    T, H, hd = (40, 2, 128) if op != "split attention" else (1, 2, 128)
    n = T if T > 1 else 5000
    q, k, v = rnd(1, T, H, hd), rnd(2, n, H, hd), rnd(3, n, H, hd)
    cos, sin = tables(T, hd)
    M = 4096 if op == "linear many rows" else 3
    a, w = rnd(5, M, 256), rnd(6, 4096, 256)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    lin, o, tab = torch.zeros(M, 4096, device="cuda"), torch.zeros_like(q), torch.zeros(2, T, hd // 2, device="cuda")
    batch = Z.PromptBatch([T], [n])
    ws = workspace(batch, H, H, hd)
    assert (ws is not None) == (op == "split attention")
    stream = torch.cuda.default_stream()
    call = {
        "rope": lambda: Z.zdit_rope_table_scaled(pos, hd, 1e4, tab[0], tab[1], stream=stream),
        "qk": lambda: Z.zdit_qk_norm_rope(q, None, o, None, None, None, cos, sin, hd, stream=stream),
        "attention": lambda: Z.zdit_prompt_attention(q, k, v, o, batch, ws, stream=stream),
        "split attention": lambda: Z.zdit_prompt_attention(q, k, v, o, batch, ws, stream=stream),
        "linear": lambda: Z.zdit_linear(a, w, lin, stream=stream),
        "linear many rows": lambda: Z.zdit_linear(a, w, lin, stream=stream),
    }[op]
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in (lin, o, tab)]
    for x in (lin, o, tab):
        x.zero_()
    torch.cuda.synchronize()
    side, graph = C.c_void_p(), C.c_void_p()
    assert rt.cudaStreamCreate(C.byref(side)) == 0
    assert rt.cudaStreamBeginCapture(side, 0) == 0  # global
    try:
        with pytest.raises(Z.ZditError, match="ZDIT_ERR_CUDA"):
            call()
    finally:
        rt.cudaStreamEndCapture(side, C.byref(graph))  # (an error: the capture was invalidated)
        rt.cudaGetLastError()
        assert rt.cudaStreamDestroy(side) == 0
    other = torch.empty(2, T, hd // 2, device="cuda")
    Z.zdit_rope_table_scaled(pos, hd, 1e4, other[0], other[1], stream=stream)
    call()
    assert Z.zdit_device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip((lin, o, tab), want))


@pytest.mark.parametrize("M,N,K", [(1, 37, 100), (9, 1, 100), (1, 1, 3), (1, 5000, 260)])
def test_linear_takes_a_single_row_of_any_stride(M, N, K):
    # the stride of a matrix with one row leads nowhere: contiguous rows of K = 100, and views
    # whose stride is smaller or larger than the row
    pad = lambda seed, rows, scale=1.0: rnd(seed, rows, K, scale=scale) if rows == 1 else \
        rnd(seed, rows, K + 12 + (4 - K) % 8, scale=scale)[:, :K]
    a, w, x = pad(1, M), pad(2, N, K ** -0.5), rnd(3, M, N, dtype=torch.float32)
    ref, e = linear_ref(a, w, None, Z.ACT_SILU, x)
    want = None
    for ld in ({K, 1, 4 * K + 1, 1 << 40} if M == 1 else {K}):
        one = torch.as_strided(a, (1, K), (ld, 1)) if M == 1 else a
        res = torch.as_strided(x, (1, N), (ld, 1)) if M == 1 else x
        o = torch.full((M, N), 9.0, device="cuda")
        Z.zdit_linear(one, w, torch.as_strided(o, (1, N), (ld, 1)) if M == 1 else o, act=Z.ACT_SILU, residual=res)
        check(o, ref, e + 2.0 ** -24 * ref.abs(), f"single row {M}x{N}x{K} ld {ld}")
        want = o if want is None else want
        assert torch.equal(o, want)


# ------------------------------------------------------------------ many rows and tokens
def many_tiles(M, N):
    """Whether a product has several row tiles and more tiles than the few-row kernel's two CTAs
    per SM: then the GEMM takes it whatever the expected times are."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return M > 160 and -(-N // 128) * -(-M // 128) > 2 * sms


# CTA pairs (M > 256): several tiles per pair, last tiles with one row or column of either CTA's
# half and none of the other's, K shorter than a slice, K that ends in either half of one
# single CTAs: M <= 256
GEMM_SHAPES = [
    (4100, 1500, 1003), (4225, 1345, 136), (8200, 600, 72), (40000, 100, 64), (5000, 1025, 5), (4700, 1152, 1),
    (9000, 520, 193), (161, 19300, 130), (250, 30001, 64), (200, 19100, 300), (256, 19001, 1),
]


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
@pytest.mark.parametrize("act,bias,res,out", [
    (Z.ACT_NONE, False, None, "f"),
    (Z.ACT_SILU, True, None, "b"),
    (Z.ACT_GELU, True, "f", "b"),
    (Z.ACT_GELU_TANH, False, "b", "f"),
])
def test_linear_many_rows(M, N, K, act, bias, res, out):
    assert many_tiles(M, N)
    test_linear(M, N, K, act, bias, res, out)


@pytest.mark.parametrize("M,N,K", [(4100, 1500, 1000), (4100, 1504, 264), (193, 20000, 256), (256, 19002, 64)])
@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
def test_linear_many_rows_residual_in_place(M, N, K, ty):
    assert many_tiles(M, N)
    test_linear_residual_in_place(M, N, K, ty)


@pytest.mark.parametrize("M,N,K", [(1, 38000, 130), (7, 24577, 300), (133, 38017, 64), (160, 45000, 72)])
@pytest.mark.parametrize("act,bias,res,out", [(Z.ACT_NONE, False, "f", "f"), (Z.ACT_GELU, True, "b", "b")])
def test_linear_few_rows_many_features(M, N, K, act, bias, res, out):
    # more CTAs than the SMs hold at once
    test_linear(M, N, K, act, bias, res, out)


@pytest.mark.parametrize("M,N,K", [(145, 2560, 512), (160, 2560, 512), (160, 300, 2563), (152, 9728, 256)])
@pytest.mark.parametrize("act,bias,res,out", [(Z.ACT_NONE, False, "f", "f"), (Z.ACT_GELU, True, "b", "b")])
def test_linear_largest_row_tiles(M, N, K, act, bias, res, out):
    test_linear(M, N, K, act, bias, res, out)


@pytest.mark.parametrize("T", [4099, 16381])  # 2 and 8 tokens a group, the last group short
@pytest.mark.parametrize("hd,rot,layout,src,norm", [
    (128, 128, Z.ROPE_HALF, "b", True),           # pairs of a lane's own, both chunks
    (128, 32, Z.ROPE_HALF, "b", True),            # pairs in another lane
    (128, 72, Z.ROPE_HALF, "b", True),            # pairs through shared memory
    (80, 80, Z.ROPE_HALF, "f", True),             # the same with lanes that hold nothing
    (128, 128, Z.ROPE_INTERLEAVED, "f", True),    # pairs inside a chunk
    (128, 30, Z.ROPE_INTERLEAVED, "b", False),    # 15 pairs
])
def test_qk_norm_rope_several_tokens_a_group(T, hd, rot, layout, src, norm):
    test_qk_norm_rope(T, 32, 8, hd, rot, src, "b", norm, layout)


@pytest.mark.parametrize("T,nq,nk,hd", [(9001, 32, 8, 64), (5003, 16, 4, 256)])  # groups of 4 and of 16 lanes
@pytest.mark.parametrize("layout", [Z.ROPE_HALF, Z.ROPE_INTERLEAVED])
def test_qk_norm_rope_several_tokens_other_groups(T, nq, nk, hd, layout):
    test_qk_norm_rope(T, nq, nk, hd, hd, "b", "b", True, layout)
    test_qk_norm_rope(T, nq, nk, hd, hd // 2 + 4, "b", "f", True, layout)


@pytest.mark.parametrize("rot", [128, 72, 64])
def test_qk_norm_rope_several_tokens_in_place(rot):
    T, nq, nk, hd = 5003, 32, 8, 128
    qkv = rnd(6, T, (nq + 2 * nk) * hd)
    before = qkv.clone()
    q, k = qkv[:, :nq * hd].view(T, nq, hd), qkv[:, nq * hd:(nq + nk) * hd].view(T, nk, hd)
    w = 1 + 0.3 * rnd(1, hd, dtype=torch.float32)
    cos, sin = tables(T, rot)
    apart = [torch.empty(T, n, hd, device="cuda", dtype=torch.bfloat16) for n in (nq, nk)]
    Z.zdit_qk_norm_rope(q, k, *apart, w, w, cos, sin, rot)
    Z.zdit_qk_norm_rope(q, k, q, k, w, w, cos, sin, rot)
    assert torch.equal(q, apart[0]) and torch.equal(k, apart[1])
    assert torch.equal(qkv[:, (nq + nk) * hd:], before[:, (nq + nk) * hd:])


@pytest.mark.parametrize("T,d,sc,first", [
    (40003, 128, None, 0),                                                              # 16 rows a CTA and step
    (20011, 22, Z.RopeScaling(Z.ROPE_SCALE_LINEAR, 4.0), 7),
    (5001, 512, Z.RopeScaling(Z.ROPE_SCALE_YARN, 4.0, 32768.0, 32.0, 1.0, 1.1386), 98304),  # 4 rows
])
def test_rope_table_scaled_several_steps_a_cta(T, d, sc, first):
    test_rope_table_scaled(T, d, 1e6, sc, first)


def test_prompt_layers_from_host_threads_at_once():
    # every operator, from threads that each have a stream, buffers and lengths of their own
    from concurrent.futures import ThreadPoolExecutor
    from threading import Barrier
    L = Layer(128, 4, 2, 64)
    runs = []
    for i, q_len in enumerate([(300, 7, 41), (1, 900), (5,), (64, 64, 2000)]):
        T = sum(q_len)
        x16 = rnd(30 + i, T, L.D)
        pos = torch.cat([torch.arange(n) for n in q_len]).to(device="cuda", dtype=torch.int32)
        buf = (torch.empty(T, 8 * 64, device="cuda", dtype=torch.bfloat16), torch.empty(T, 32, device="cuda"),
               torch.empty(T, 32, device="cuda"), torch.empty(T, 4, 64, device="cuda", dtype=torch.bfloat16),
               workspace(Z.PromptBatch(q_len), 4, 2, 64))
        x = x16.float()
        alone = torch.empty_like(x)
        L.run(x, x16, pos, q_len, alone, buf)
        runs.append((x, x16, pos, q_len, buf, alone, [torch.zeros_like(x) for _ in range(50)]))
    torch.cuda.synchronize()
    start = Barrier(len(runs), timeout=60)

    def work(run):
        x, x16, pos, q_len, buf, alone, outs = run
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            start.wait()
            for o in outs:
                L.run(x, x16, pos, q_len, o, buf)
        stream.synchronize()
        return all(torch.equal(o, alone) for o in outs)

    with ThreadPoolExecutor(len(runs)) as pool:
        assert all(pool.map(work, runs))
    assert Z.zdit_device_status() == 0
