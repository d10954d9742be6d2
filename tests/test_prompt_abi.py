"""CPU checks of the prompt operators: every refusal happens on the host before a launch,
and the workspace sizing follows the split rule's contract.  No call reaches a GPU."""
import ctypes as C
import math

import pytest
import torch

import stream_diffusion_transformer_s3_b200 as Z

P = 1 << 20  # a 16-byte aligned stand-in for a device address
INVALID, SHAPE, ALIGN, WORKSPACE = -1, -2, -3, -4


def i32(*v):
    return (C.c_int32 * len(v))(*v)


# ------------------------------------------------------------------ rotary tables
def rope(pos=P, T=4, d=64, theta=1e4, sc=None, cos=P, sin=P):
    return Z.lib().zdit_rope_table_scaled(pos, T, d, theta, C.byref(sc) if sc is not None else None, cos, sin, None)


@pytest.mark.parametrize("kw,code", [
    (dict(pos=None), INVALID), (dict(cos=None), INVALID), (dict(sin=None), INVALID), (dict(T=-1), INVALID),
    (dict(theta=0.0), INVALID), (dict(theta=0.5), INVALID), (dict(theta=math.inf), INVALID),
    (dict(theta=math.nan), INVALID), (dict(d=0), SHAPE), (dict(d=63), SHAPE), (dict(d=514), SHAPE),
    (dict(cos=P + 4), ALIGN), (dict(sin=P + 8), ALIGN), (dict(pos=P + 2), ALIGN),
    (dict(sc=Z.RopeScaling(4)), INVALID), (dict(sc=Z.RopeScaling(-1)), INVALID),
    (dict(sc=Z.RopeScaling(Z.ROPE_SCALE_LINEAR, 0.5)), INVALID),
    (dict(sc=Z.RopeScaling(Z.ROPE_SCALE_LINEAR, math.nan)), INVALID),
    (dict(sc=Z.RopeScaling(Z.ROPE_SCALE_NONE, magnitude=0.0)), INVALID),
    (dict(sc=Z.RopeScaling(Z.ROPE_SCALE_YARN, 4.0, 0.0)), INVALID),
    (dict(sc=Z.RopeScaling(Z.ROPE_SCALE_YARN, 4.0, 4096.0, 1.0, 1.0)), INVALID),
    (dict(sc=Z.RopeScaling(Z.ROPE_SCALE_YARN, 4.0, 4096.0, 32.0, -1.0)), INVALID),
    (dict(sc=Z.RopeScaling(Z.ROPE_SCALE_NTK, 4.0), d=2), SHAPE),
    (dict(T=0), 0),
])
def test_rope_table_scaled_refusals(kw, code):
    assert rope(**kw) == code


# ------------------------------------------------------------------ query / key norm and rotation
def qk_args(**kw):
    hd = kw.get("head_dim", 128)
    nq, nk = kw.get("n_q", 4), kw.get("n_k", 2)
    a = Z.QkNormRopeArgs(T=4, n_q=4, n_k=2, head_dim=128, in_dtype=0, out_dtype=0, eps=1e-6, rotary_dim=128, layout=1)
    a.q, a.q_out = Z.Heads(P, nq * hd, hd), Z.Heads(2 * P, nq * hd, hd)
    a.k, a.k_out = Z.Heads(3 * P, nk * hd, hd), Z.Heads(4 * P, nk * hd, hd)
    a.cos = a.sin = a.w_q = a.w_k = P
    for n, v in kw.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(n_q=0), INVALID), (dict(n_k=-1), INVALID), (dict(q=Z.Heads(None, 512, 128)), INVALID),
    (dict(k_out=Z.Heads(None, 256, 128)), INVALID), (dict(in_dtype=2), INVALID), (dict(out_dtype=-1), INVALID),
    (dict(layout=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(cos=None), INVALID),
    (dict(head_dim=4), SHAPE), (dict(head_dim=100), SHAPE), (dict(head_dim=264), SHAPE), (dict(rotary_dim=127), SHAPE),
    (dict(rotary_dim=130), SHAPE), (dict(rotary_dim=-2), SHAPE), (dict(q_out=Z.Heads(P, 256, 128)), SHAPE),
    (dict(q_out=Z.Heads(P, 512, 64)), SHAPE), (dict(q=Z.Heads(P, -512, 128)), SHAPE),
    (dict(q=Z.Heads(P + 8, 512, 128)), ALIGN), (dict(q=Z.Heads(P, 516, 128)), ALIGN),
    (dict(k_out=Z.Heads(P, 512, 132)), ALIGN), (dict(w_q=P + 4), ALIGN), (dict(cos=P + 4), ALIGN),
    (dict(T=1 << 33), SHAPE), (dict(T=0), 0),
    # one buffer for input and output, but not element by element
    (dict(q_out=Z.Heads(P, 1024, 128)), INVALID), (dict(q_out=Z.Heads(P, 512, 128), out_dtype=1), INVALID),
    (dict(k_out=Z.Heads(3 * P, 128, 512)), INVALID),
])
def test_qk_norm_rope_refusals(kw, code):
    assert Z.lib().zdit_qk_norm_rope(C.byref(qk_args(**kw)), None) == code


@pytest.mark.parametrize("kw", [
    dict(k_out=Z.Heads(2 * P, 256, 128)), dict(q_out=Z.Heads(3 * P, 512, 128)), dict(k_out=Z.Heads(P, 256, 128)),
])
def test_qk_norm_rope_refuses_one_buffer_for_two_heads(kw):
    # both outputs, or an output and the other input, in one place
    assert Z.lib().zdit_qk_norm_rope(C.byref(qk_args(**kw)), None) == INVALID


def test_rope_table_scaled_refuses_one_buffer_for_both_tables():
    assert rope(cos=P, sin=P, T=4) == INVALID


def test_qk_norm_rope_refuses_null():
    assert Z.lib().zdit_qk_norm_rope(None, None) == INVALID


def test_qk_norm_rope_allows_a_null_key_side_and_tables():
    # nothing rotates and there are no keys: every check passes (no rows, so nothing runs)
    a = qk_args(T=0, n_k=0, k=Z.Heads(), k_out=Z.Heads(), rotary_dim=0, cos=None, sin=None, w_k=None)
    assert Z.lib().zdit_qk_norm_rope(C.byref(a), None) == 0


# ------------------------------------------------------------------ attention
def pa(q_len=(3, 5), kv_len=None, kv_start=None, H=8, Hkv=2, hd=128, **kw):
    a = Z.PromptAttentionArgs(batch=len(q_len), q_len=i32(*q_len), n_heads=H, n_kv_heads=Hkv, head_dim=hd, causal=1,
                              scale=0.0)
    if kv_len is not None:
        a.kv_len = i32(*kv_len)
    if kv_start is not None:
        a.kv_start = i32(*kv_start)
    a.q, a.o = Z.Heads(P, H * hd, hd), Z.Heads(2 * P, H * hd, hd)
    a.k, a.v = Z.Heads(3 * P, max(Hkv, 1) * hd, hd), Z.Heads(4 * P, max(Hkv, 1) * hd, hd)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def attn(a, ws=None, n=0):
    return Z.lib().zdit_prompt_attention(C.byref(a), ws, n, None)


@pytest.mark.parametrize("a,code", [
    (dict(batch=0), SHAPE), (dict(batch=129), SHAPE), (dict(q_len=(-1, 2)), SHAPE), (dict(kv_len=(-1, 2)), SHAPE),
    (dict(kv_start=(-1, 2)), SHAPE), (dict(kv_start=(1 << 30, 0), kv_len=(3, 3)), SHAPE), (dict(H=8, Hkv=3), SHAPE),
    (dict(H=65, Hkv=1), SHAPE), (dict(Hkv=0), SHAPE), (dict(hd=96), SHAPE), (dict(causal=2), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
    (dict(q=Z.Heads(None, 1024, 128)), INVALID), (dict(v=Z.Heads(None, 256, 128)), INVALID),
    (dict(q=Z.Heads(P, 64, 128)), SHAPE), (dict(k=Z.Heads(P, 256, 64)), SHAPE),
    (dict(k=Z.Heads(P, 1 << 39, 128)), SHAPE), (dict(o=Z.Heads(2 * P, 512, 128)), SHAPE),
    (dict(q=Z.Heads(P + 8, 1024, 128)), ALIGN), (dict(k=Z.Heads(P, 260, 128)), ALIGN),
    (dict(o=Z.Heads(2 * P, 1028, 128)), ALIGN), (dict(q_len=(0, 0)), 0),
    (dict(o=Z.Heads(P, 1024, 128)), INVALID), (dict(o=Z.Heads(4 * P, 1024, 128)), INVALID),
])
def test_prompt_attention_refusals(a, code):
    kw = dict(a)
    batch = kw.pop("batch", None)
    args = pa(**kw)
    if batch is not None:
        args.q_len = i32(*([1] * max(batch, 1)))
        args.batch = batch
    assert attn(args) == code


def test_prompt_attention_refuses_null():
    assert Z.lib().zdit_prompt_attention(None, None, 0, None) == INVALID
    a = pa()
    a.q_len = None
    assert attn(a) == INVALID
    assert Z.lib().zdit_prompt_attention_workspace_bytes(None) == 0


def test_prompt_attention_workspace():
    size = lambda a: Z.lib().zdit_prompt_attention_workspace_bytes(C.byref(a))
    assert size(pa((64, 9))) == 0                          # short prompts: nothing to split
    assert size(pa((16384,), H=32, Hkv=8)) == 0            # the rows fill the GPU
    assert size(pa((1,), Hkv=3)) == 0                      # invalid
    long = pa((1,), kv_len=(32768,), H=32, Hkv=8)
    need = size(long)
    assert need >= 2 * 32 * (128 * 4 + 8)                  # at least two parts of 32 rows
    assert attn(long) == WORKSPACE
    assert attn(long, P, need - 1) == WORKSPACE
    assert attn(long, P + 128, need) == ALIGN
    # parts are bounded by what fills the GPU, whatever the lengths
    assert size(pa((200,) * 8, kv_len=(200000,) * 8, H=32, Hkv=8)) < 1 << 30


# ------------------------------------------------------------------ linear
def lin(**kw):
    a = Z.LinearArgs(M=4, N=8, K=16, a=P, lda=16, w=2 * P, ldw=16, out=3 * P, ld_out=8)
    for n, v in kw.items():
        setattr(a, n, v)
    return Z.lib().zdit_linear(C.byref(a), None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(act=4), INVALID), (dict(act=-1), INVALID), (dict(out_dtype=2), INVALID),
    (dict(residual=P, ld_residual=8, residual_dtype=3), INVALID), (dict(a=None), INVALID), (dict(w=None), INVALID),
    (dict(out=None), INVALID), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(N=9), SHAPE), (dict(lda=8), SHAPE),
    (dict(ldw=8), SHAPE), (dict(residual=P, ld_residual=7), SHAPE), (dict(M=(1 << 30) + 1), SHAPE),
    (dict(lda=20), ALIGN), (dict(ldw=20), ALIGN), (dict(a=P + 8), ALIGN), (dict(w=P + 2), ALIGN),
    (dict(bias=P + 2), ALIGN), (dict(out=3 * P + 1), ALIGN), (dict(out=3 * P + 2, out_dtype=1), ALIGN),
    (dict(residual=P + 2, ld_residual=8, residual_dtype=1), ALIGN), (dict(M=0), 0), (dict(M=0, a=None, out=None), 0),
    (dict(out=P), INVALID), (dict(out=2 * P), INVALID),
    (dict(residual=3 * P, ld_residual=8, residual_dtype=1), INVALID), (dict(residual=3 * P, ld_residual=16), INVALID),
])
def test_linear_refusals(kw, code):
    assert lin(**kw) == code


def test_linear_refuses_null():
    assert Z.lib().zdit_linear(None, None) == INVALID


# ------------------------------------------------------------------ the binding's own checks
def test_binding_refuses_what_the_structs_cannot_carry():
    b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        Z.PromptBatch([1, 2], [3])
    batch = Z.PromptBatch([3], [5], [2])
    assert (batch.q_rows, batch.kv_rows) == (3, 7)
    q, k = b16(3, 4, 128), b16(7, 2, 128)
    with pytest.raises(ValueError):
        Z.zdit_prompt_attention(q.float(), k, k, q, batch)           # type
    with pytest.raises(ValueError):
        Z.zdit_prompt_attention(q, k[:6], k[:6], q, batch)           # fewer key rows than the batch names
    with pytest.raises(ValueError):
        Z.zdit_prompt_attention(q[:2], k, k, q, batch)               # fewer query rows
    with pytest.raises(ValueError):
        Z.zdit_prompt_attention(q, k, k[:, :1], q, batch)            # k and v differ
    with pytest.raises(ValueError):
        Z.zdit_prompt_attention(q.transpose(1, 2), k, k, q, batch)   # last axis strided
    a, w = b16(4, 16), b16(8, 16)
    with pytest.raises(ValueError):
        Z.zdit_linear(a.float(), w, b16(4, 8))
    with pytest.raises(ValueError):
        Z.zdit_linear(a, w, b16(4, 9))
    with pytest.raises(ValueError):
        Z.zdit_linear(a, w, b16(4, 8), bias=torch.zeros(7))
    with pytest.raises(ValueError):
        Z.zdit_linear(a, w, b16(4, 8).half())
    with pytest.raises(ValueError):
        Z.zdit_rope_table_scaled(torch.zeros(3), 64, 1e4, torch.zeros(3, 32), torch.zeros(3, 32))
    with pytest.raises(ValueError):
        Z.zdit_qk_norm_rope(q, k, q, k, None, None, torch.zeros(3, 64), torch.zeros(3, 64), 128)  # rows differ


def test_binding_refuses_a_workspace_with_less_memory_than_elements():
    # an expanded or strided tensor names more bytes than it holds from its first on
    b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    q, k = b16(1, 32, 128), b16(8192, 8, 128)
    batch = Z.PromptBatch([1], [8192])
    need = Z.prompt_attention_workspace_bytes(batch, 32, 8, 128)
    assert need > 0
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(2 * need, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            Z.zdit_prompt_attention(q, k, k.clone(), q.clone(), batch, ws)


@pytest.mark.parametrize("lens", [
    dict(q_len=[1 << 32]), dict(q_len=[1], kv_len=[(1 << 32) + 5]), dict(q_len=[1], kv_len=[5], kv_start=[1 << 32]),
    dict(q_len=[1], kv_len=[5], kv_start=[-(1 << 32)]), dict(q_len=[1 << 31]),
])
def test_batch_lengths_past_32_bits_are_refused(lens):
    # (kept modulo 2^32 they would be other rows)
    with pytest.raises(ValueError, match="PromptBatch"):
        Z.PromptBatch(**lens)


def test_batch_cannot_change_after_its_rows_were_counted():
    # the rows a batch needs are counted once; the library reads the lengths on every call
    b = Z.PromptBatch([1, 2], [5, 6], [0, 9])
    assert (list(b.q_len), list(b.kv_len), list(b.kv_start)) == ([1, 2], [5, 6], [0, 9])
    for name in ("q_len", "kv_len", "kv_start"):
        with pytest.raises(TypeError):
            getattr(b, name)[0] = 1000
        with pytest.raises(AttributeError):
            setattr(b, name, [1000, 1000])
    for name in ("batch", "q_rows", "kv_rows"):
        with pytest.raises(AttributeError):
            setattr(b, name, 1)
    assert (b.batch, b.q_rows, b.kv_rows) == (2, 3, 15)
    plain = Z.PromptBatch([3, 4])
    assert plain.kv_len is None and plain.kv_start is None and plain.kv_rows == 7


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_batch_copies_own_their_lengths(how):
    # (addresses of the first one's arrays would outlive it, or mean nothing in another process)
    import copy
    import pickle
    b = Z.PromptBatch([1, 2], [500, 600], [0, 900])
    c = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda x: pickle.loads(pickle.dumps(x))}[how](b)
    old, new = b.args(4, 2, 128, True, 0.0), c.args(4, 2, 128, True, 0.0)
    for name in ("q_len", "kv_len", "kv_start"):
        x, y = getattr(old, name), getattr(new, name)
        assert C.addressof(x.contents) != C.addressof(y.contents)
        assert x[:2] == y[:2] == list(getattr(c, name))
    assert (c.batch, c.q_rows, c.kv_rows) == (2, 3, 1500)
